// chunk_tc.cu -- attention of query rows to a paged cache, bf16 or e4m3, on
// sm_100a tensor cores: causal chunks of new tokens (ragged, windowed, from
// one token to whole prompts), and the rows of a draft tree over an e4m3
// cache followed by the tree's own keys.
//
//   o = sum_j e^{x_j} v_j / sum_j e^{x_j},  x_j = scale * q.k_j over the keys
//   a row sees; one pass with a running maximum m and sum l of 2^{x - m}.
//
// Items.  The G query heads of a KV head share its keys, so the rows of a
// (sequence, KV head) are packed (chunk: r = t*G + g, tree: r = g*T + t) and
// cut into items of up to 256 rows: two 128-row MMA tiles that share every
// K/V tile they read (one tile when at most 128 rows are left).  An item's
// keys come in tiles of 128.
//
// Schedule (chunk_plan.cuh).  Lengths are known to the device only, so every
// CTA (one per SM) computes the work of all items and takes an equal,
// contiguous range of the whole: long axes are split over as many CTAs as it
// takes and ragged batches balance, without a plan kernel or a host copy.  An
// item that lies in one CTA's range is finished there; one that crosses a
// border leaves normalised fp32 partials and their lse, at most two per CTA
// (its first and its last item), which chunk_merge_kernel joins.  Nothing
// depends on the order in which CTAs run.
//
// Warps: 0 TMA producer of K, 1 MMA issuer, 2 TMA producer of V, 3 fixer of
// partly visible V tiles (bf16 caches), 4-7 and 8-11 two softmax groups (one
// row per thread), 12-15 and 16-19 loaders of K and of V (e4m3 caches).  With
// two row tiles group g owns tile g and runs every key tile; with one, group g
// runs the key tiles j = g mod 2 into an accumulator of its own and the two are
// merged at the end (the lse merge of two key ranges).  Steps s of an item:
// group s & 1, key tile s >> (two row tiles); MMA order QK_0 QK_1 [PV_0 QK_2]
// [PV_1 QK_3] ..., P*V in two halves of the keys, the first while the softmax
// group works on the second (prefill 990 -> 963 us).
//
// e4m3 caches.  TMA leaves a tile's codes in the upper half of its stage; a
// loader reads its row into registers and writes it back over the whole stage
// as the swizzled f16 tile the MMAs read, so that codes need no buffers of
// their own and the rings prefetch as deep as for bf16.  (Loads straight into
// registers, one tile ahead, took 5 us a tile: a warp's waits on them cover
// younger loads too, so that each tile waited for the next one's.)  The MMAs
// run in f16: every code is one of f16's numbers, and two conversions and two
// products make four of them where bf16 takes ten instructions.  A tile's rows
// are brought to its largest scale E where none lies more than 15 octaves below
// it (K; no code leaves f16's numbers) or 4 (V), and 2^(E - 127) goes to the
// scores, or for V to the weights.  Tiles of rows further apart keep the codes
// as they are, and each key's scale byte goes to its own score or weight (8
// trees with every tile such: 571 us against 287).  The weights P stand relative
// to the running maximum of x + scale of V, kept as m_run + e_run, so that they
// stay in f16's range beside tiles of large values or of zeros; from E alone the
// maximum comes out 4 octaves too high at most, which is why V's limit is low.
// Rows of queries and of the tree are scaled by powers of two into f16 (the
// tree's by the tile or by the row, as above), which holds bf16's 8 bits down to
// 2^-28 of the row's largest value.
//
// Measured (B200, 1965 MHz, at the power cap in long runs): prefill of 4096
// tokens behind 12288, 32 heads over 8: 0.96-1.00 ms, 0.96-1.00 PFLOP/s, 0.6 of
// cuBLAS's rate.  A pair of 128 x 128 tiles took 3.7 k cycles against 2048 of MMA
// before the second sum (below), 3.8 k by the time since: the chain of a group is
// its softmax (1.9 k), the MMAs of the next scores behind it (1.0 k) and hand-overs,
// and two groups fill the MMAs to 55 %; issuing eight MMAs takes 70 cycles, and no
// pipe is above 45 %.  Decode of 16 sequences, bf16:
// 208-213 us, 0.90-0.92 of the measured copy.  A 68-node tree over e4m3 keys,
// 8 x 32 heads: 292-315 us, 2.6 TB/s of codes: 3.0 k cycles a 128-key tile, of which
// the conversion's traffic in shared memory beside the MMAs' own costs 0.6 k
// (without it 2.4 k).
//
// Tensor memory: S[g] columns 128g.. (fp32 scores; P as 16-bit pairs over its
// last 64), O[g] columns 256 + gD...  P is rounded to bf16 (e4m3 caches: f16)
// for the tensor cores, by 2^-8 of a weight at most (f16: 2^-11); its sums, the
// maximum and O stay in fp32.  The running maximum moves only when it grew by
// more than 2^8, so that the largest weight is a rounded one too: with bf16 O is
// divided by the sum of what P holds, and a weight's rounding reaches the result
// only by as much as its V differs from the result (rows with a few heavy keys,
// scores of 8 sigma: worst row 4.1e-3 -> 2.4e-3 off, of which 2.4e-3 the output's
// own rounding).  The lse takes the sum of the unrounded weights.  The second sum
// costs the prefill 3 % (938 -> 966 us), ragged chunks 4-5 %, decode 2 %; made
// behind the hand-over of P, or from weights cut off instead of rounded, the same.
//
// Keys a row does not see: scores are set to -inf, and rows of V that no row
// of the item may see are zeroed in shared memory (a cache row behind the
// last key may hold anything).  A V row that some rows see and others do not
// loses its infinities and NaN there (0 * inf would reach the others); the rows
// that see it get them added to their columns at the end, from the cache.  (A
// row of an e4m3 cache is NaN as a whole: zeroed, and the rows that see it NaN.)
#include "chunk_plan.cuh"

namespace hta {

namespace {

// NaN words and scale bytes of the tiles in flight: K of tile p is there at the earliest when
// the softmax of tile p - NK - 2 is done, so NK + 2 places are enough
constexpr int kPoisonRing = 6;

template <int D, bool Q8, bool ONE>
struct Cfg {
    // ring depths; with ONE row tile an item the second Q tile makes another stage
    static constexpr int NK = D == 128 ? 3 : 4;
    static constexpr int NV = (D == 128 ? 2 : 4) + (ONE ? 1 : 0);
    static constexpr int HALVES = D / 64;                   // 64-column swizzle boxes
    static constexpr int BOX = 128 * 64 * 2;
    static constexpr int TILE = 128 * D * 2;
    static constexpr int RAW = 128 * D;                     // a tile's codes, in the upper half of its stage
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = (ONE ? 1 : 2) * TILE;
    static constexpr int OFF_V = OFF_K + NK * TILE;
    static constexpr int OFF_BAR = OFF_V + NV * TILE;
    // q_full, q_empty, o_full, o_empty, drain, k_full[NK], k_empty[NK], k_raw[NK], v_full[NV], v_empty[NV],
    // v_raw[NV], s_full[2], p_ready[2][2] (halves of the keys).  x_raw: a tile as TMA left it; x_full: ready for the MMAs
    static constexpr int NUM_BARS = 5 + 3 * NK + 3 * NV + 6;
    static_assert(kPoisonRing >= NK + 2, "see kPoisonRing");
    static constexpr int OFF_POISON = (OFF_BAR + NUM_BARS * 8 + 15) / 16 * 16;   // [kPoisonRing][4] words
    static constexpr int OFF_MISC = OFF_POISON + kPoisonRing * 16;   // tmem base, abort; Start
    static_assert(sizeof(Start) <= 80, "room of the plan's result");
    static constexpr int OFF_PARENT = OFF_MISC + 96;                 // parent + 1 of each node, a byte (trees)
    static constexpr int OFF_SCALE = OFF_PARENT + kTMax;             // per tile in flight: scale bytes of K and of V
    static constexpr int OFF_SCALE_V = OFF_SCALE + (Q8 ? kPoisonRing * 256 : 0);   // per V stage: V's once more, for the V loaders
    static constexpr int OFF_WALK = OFF_SCALE_V + (Q8 ? NV * 128 : 0);     // walks: softmax groups, K and V loaders
    static constexpr int WALK_BYTES = 128;
    static constexpr int OFF_EXP = OFF_WALK + (Q8 ? 3 : 1) * WALK_BYTES;   // per tile in flight: E of K, E of V
    static constexpr int OFF_RED = OFF_EXP + (Q8 ? kPoisonRing * 8 : 0);   // [2][4] words: a maximum over a loader set
    static constexpr int SMEM_ALLOC = OFF_RED + (Q8 ? 32 : 0);
    static constexpr int OFF_XCH = OFF_Q;                   // [8][128] floats: Q has been read by then
    static constexpr int OFF_PLAN = OFF_K;                  // int64 [kPlanUnits], before the first copy
    static constexpr int THREADS = Q8 ? 640 : 384;
    // registers per thread; the launch allots LAUNCH_REGS to each
    static constexpr int LAUNCH_REGS = Q8 ? 96 : 168;
    static constexpr int REGS_SOFTMAX = Q8 ? 120 : 224;
    static constexpr int REGS_LOAD = 88;
    static constexpr int REGS_OTHER = Q8 ? 64 : 56;
    static_assert(256 * REGS_SOFTMAX + (Q8 ? 256 * REGS_LOAD : 0) + 128 * REGS_OTHER <= THREADS * LAUNCH_REGS,
                  "register split must fit the launch allocation");
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static constexpr uint32_t F16 = Q8 ? ~((1u << 7) | (1u << 10)) : ~0u;   // (format 1 of A and B: bf16, 0: f16)
    static constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, 128, false) & F16;
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, true) & F16;
    static constexpr int COL_S = 0, COL_O = 256;
};

constexpr int kWarpK = 0, kWarpMma = 1, kWarpV = 2, kWarpFix = 3, kWarpSoftmax = 4, kWarpLoad = 12;

// ------------------------------------------------------------ small helpers
__device__ __forceinline__ bool bar_or(int id, int n, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "bar.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(id), "r"(n), "r"(pred ? 1u : 0u) : "memory");
    return r != 0;
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unf2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// 2^d in f16 (d <= 0; 0 below 2^-24), twice
__device__ __forceinline__ uint32_t f16_pow2(int d) {
    const uint32_t h = d >= -14 ? static_cast<uint32_t>(15 + d) << 10 : d >= -24 ? 1u << (24 + d) : 0u;
    return h | (h << 16);
}
// four e4m3 codes times an f16 pair `mult`, as two f16 pairs
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t w, uint32_t mult) {
    uint2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 a, b;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 a, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 b, hi;\n\t"
        "mul.rn.f16x2 %0, a, %3;\n\t"
        "mul.rn.f16x2 %1, b, %3;\n\t}"
        : "=r"(r.x), "=r"(r.y) : "r"(w), "r"(mult));
    return r;
}
__device__ __forceinline__ float pow2(int d) { return __uint_as_float(static_cast<uint32_t>(127 + d) << 23); }
// largest |bf16| bit pattern of eight values and `big`
__device__ __forceinline__ uint32_t max_bits(uint4 u, uint32_t big) {
    big = __vmaxu2(__vmaxu2(big, u.x & 0x7fff7fffu), __vmaxu2(u.y & 0x7fff7fffu, u.z & 0x7fff7fffu));
    return __vmaxu2(big, u.w & 0x7fff7fffu);
}
// eight bf16 values with infinities and NaN as 0
__device__ __forceinline__ uint32_t finite(uint32_t x) {
    return ((x & 0x7f80u) == 0x7f80u ? 0u : x & 0xffffu) | ((x & 0x7f800000u) == 0x7f800000u ? 0u : x & 0xffff0000u);
}
__device__ __forceinline__ uint4 finite(uint4 u) { return make_uint4(finite(u.x), finite(u.y), finite(u.z), finite(u.w)); }
__device__ __forceinline__ uint32_t halves_max(uint32_t m) { return max(m & 0xffffu, m >> 16); }
// eight bf16 values times `mul`, as f16
__device__ __forceinline__ uint4 to_f16(uint4 u, float mul) {
    return make_uint4(pack_f16x2(bf16_lo(u.x) * mul, bf16_hi(u.x) * mul), pack_f16x2(bf16_lo(u.y) * mul, bf16_hi(u.y) * mul),
                      pack_f16x2(bf16_lo(u.z) * mul, bf16_hi(u.z) * mul), pack_f16x2(bf16_lo(u.w) * mul, bf16_hi(u.w) * mul));
}
// the shift that brings a largest bit pattern into [2^14, 2^15), at most `most`
__device__ __forceinline__ int f16_shift(uint32_t big, int most) {
    return max(min(14 - (static_cast<int>(big >> 7) - 127), most), -113);
}

template <int N> struct Int { static constexpr int value = N; };

// Octaves between a tile's largest and least row scale up to which its rows are
// brought to the largest (see the head of this file)
constexpr int kSpreadK = 15, kSpreadV = 4;
constexpr int kEach = 256;          // bit of a tile's scale: its rows keep their own

// registers of a tensor-memory load that has been waited for
__device__ __forceinline__ void pin(uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// NaN if any operand is (a NaN score must not get lost in the clamps below)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

}  // namespace

// ------------------------------------------------------------------- kernel
template <int D, bool Q8, bool ONE>
__global__ void __launch_bounds__(Cfg<D, Q8, ONE>::THREADS, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                const __grid_constant__ ChunkParams p) {
    using C = Cfg<D, Q8, ONE>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (smem_u32(smem) & 1023u) {                   // (the swizzled tiles need it; every slot is left empty)
        if (threadIdx.x == 0) {
            raise_status(p.status, kStatusInternal);
            p.heads[2 * blockIdx.x].rows = p.heads[2 * blockIdx.x + 1].rows = 0;
        }
        return;
    }

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *q_full = bars, *q_empty = bars + 1, *o_full = bars + 2, *o_empty = bars + 3, *drain = bars + 4;
    uint64_t *k_full = bars + 5, *k_empty = k_full + C::NK, *k_raw = k_empty + C::NK;
    uint64_t *v_full = k_raw + C::NK, *v_empty = v_full + C::NV, *v_raw = v_empty + C::NV;
    uint64_t *s_full = v_raw + C::NV, *p_ready = s_full + 2;
    uint32_t *s_poison = reinterpret_cast<uint32_t *>(smem + C::OFF_POISON);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    Start *s_start = reinterpret_cast<Start *>(smem + C::OFF_MISC + 16);
    uint8_t *s_parent = smem + C::OFF_PARENT;       // (parent + 1)
    uint8_t *s_scale = smem + C::OFF_SCALE;
    int2 *s_exp = reinterpret_cast<int2 *>(smem + C::OFF_EXP);

    if (threadIdx.x == 0) {
        mbar_init(q_full, 8);                       // one arrive per softmax warp
        mbar_init(q_empty, 1);
        mbar_init(o_full, 1);
        mbar_init(o_empty, 8);
        // (one arrive per loader warp, by TMA or by the fixer)
        for (int i = 0; i < C::NK; ++i) { mbar_init(k_full + i, Q8 ? 4 : 1); mbar_init(k_empty + i, 1); mbar_init(k_raw + i, 1); }
        for (int i = 0; i < C::NV; ++i) { mbar_init(v_full + i, Q8 ? 4 : 1); mbar_init(v_empty + i, 1); mbar_init(v_raw + i, 1); }
        for (int i = 0; i < 2; ++i) mbar_init(s_full + i, 1);
        for (int i = 0; i < 4; ++i) mbar_init(p_ready + i, 4);
        mbar_init(drain, 1);
        *s_abort = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < kPoisonRing * 4) s_poison[threadIdx.x] = 0;
    if (warp == kWarpMma) {
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    // lengths, queries and the cache may come from the previous kernel
    asm volatile("griddepcontrol.wait;" ::: "memory");
    plan_start(p, reinterpret_cast<long long *>(smem + C::OFF_PLAN), s_start);
    fence_proxy_async();                            // the plan's scratch becomes the K ring
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    auto warp_wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, s_abort, p.status));
    };

    Walk w;
    const int bs = p.cache.block_size, bsh = __ffs(bs) - 1;

    if (warp == kWarpK || warp == kWarpV) {
        // ---------------------------------------------------- TMA producers
        regs_dec<C::REGS_OTHER>();
        const bool is_k = warp == kWarpK;
        const int ns = is_k ? C::NK : C::NV;
        uint8_t *ring = smem + (is_k ? C::OFF_K : C::OFF_V);
        // K tiles of a bf16 cache go straight to the MMAs, the others by the loaders or the fixer
        uint64_t *full = is_k ? (Q8 ? k_raw : k_full) : v_raw, *empty = is_k ? k_empty : v_empty;
        const CUtensorMap *map = is_k ? &tm_k : &tm_v, *tree_map = is_k ? &tm_kt : &tm_vt;
        if (lane == 0) tma_prefetch_desc(map);
        const int nb = 128 >> bsh;
        int st = 0, ph = 1, issued = 0;
        bool ok = true;
        w.start(p, s_start);
        while (ok && w.next(p)) {
            const int32_t *row = p.cache.block_table + static_cast<size_t>(w.cur_b) * p.cache.max_blocks;
            const int first = w.it.lo >> bsh, last = (w.it.hi - 1) >> bsh;
            // blocks outside the item's keys are not looked up: their rows
            // repeat a block inside (masked, and zeroed in V)
            auto fetch = [&](int j) {
                return lane < nb && w.it.hi > 0 && j < w.it.cache_tiles
                           ? row[min(max((w.key0(j) >> bsh) + lane, first), last)] : 0;
            };
            int id = fetch(w.j0);
            for (int j = w.j0; j < w.j1; ++j) {
                if (!warp_wait(empty + st, ph)) { ok = false; break; }
                uint8_t *stage = ring + st * C::TILE;
                if (j >= w.it.cache_tiles) {            // rows of the tree (behind them: other trees', or zeros)
                    if (Q8 && lane == 0) {
                        mbar_arrive_expect_tx(full + st, C::TILE);
                        const int y = (w.cur_b * p.Hkv + w.cur_kvh) * p.N + (j - w.it.cache_tiles) * 128;
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h) tma_load_2d(stage + h * C::BOX, tree_map, full + st, h * 64, y);
                    }
                } else if (w.it.hi == 0) {              // nothing to read: a wholly masked tile
                    if (lane == 0) mbar_arrive(full + st);
                } else {
                    if (lane == 0) mbar_arrive_expect_tx(full + st, Q8 ? C::RAW + (is_k ? 256 : 128) : C::TILE);
                    __syncwarp();
                    if (lane < nb) {
                        int n = id;
                        if (n < 0 || n >= p.cache.num_blocks) {
                            raise_status(p.status, kStatusBadBlock);
                            n = 0;
                        }
                        const int y = (n * p.Hkv + w.cur_kvh) << bsh;
                        if constexpr (Q8) {
                            tma_load_2d(stage + C::TILE - C::RAW + (lane << bsh) * D, map, full + st, 0, y);
                            if (is_k) {                 // (V's scale bytes too: see the K loaders)
                                uint8_t *sc = s_scale + issued % kPoisonRing * 256 + (lane << bsh);
                                bulk_load(sc, p.cache.k_scale + y, bs, full + st);
                                bulk_load(sc + 128, p.cache.v_scale + y, bs, full + st);
                            } else {
                                bulk_load(smem + C::OFF_SCALE_V + st * 128 + (lane << bsh), p.cache.v_scale + y, bs, full + st);
                            }
                        } else {
#pragma unroll
                            for (int h = 0; h < C::HALVES; ++h)
                                tma_load_2d(stage + h * C::BOX + (lane << bsh) * 128, map, full + st, h * 64, y);
                        }
                    }
                }
                id = fetch(j + 1);
                ++issued;
                if (++st == ns) { st = 0; ph ^= 1; }
            }
        }
        __syncwarp();
        if (lane == 0 && *s_abort)                      // let the copies in flight land
            for (int i = max(0, issued - ns); i < issued; ++i) mbar_wait(full + i % ns, (i / ns) & 1);
        __syncwarp();
    } else if (warp == kWarpFix) {
        // ------------------- partly visible V tiles of a bf16 cache, in place
        // (every tile passes here, so that the phases of v_full follow the ring)
        regs_dec<C::REGS_OTHER>();
        if constexpr (!Q8) {
            int pos = 0;
            bool ok = true;
            w.start(p, s_start);
            while (ok && w.next(p)) {
                for (int j = w.j0; j < w.j1; ++j, ++pos) {
                    const int st = pos % C::NV;
                    if (!warp_wait(v_raw + st, pos / C::NV)) { ok = false; break; }
                    if (!w.partial(j)) {
                        if (lane == 0) mbar_arrive(v_full + st);
                        continue;
                    }
                    uint8_t *sv = smem + C::OFF_V + st * C::TILE;
                    const int a = w.it.lo - w.key0(j), z = w.it.hi - w.key0(j);   // live rows [a, z)
                    // A row per lane, four rounds, rounds of rows that every query row sees
                    // left out (what such a row holds is everybody's).
                    for (int g = 0; g < 4; ++g) {
                        const int r = g * 32 + lane, key = w.key0(j) + r;
                        uint8_t *rp = sv + r * 128;
                        const bool live = r >= a && r < z;
                        const bool some = live && (key < w.it.all_lo || key >= w.it.all_hi);
                        uint32_t word = 0;
                        if (__any_sync(0xffffffffu, some || !live)) {
                            uint32_t big = 0;           // bit 15 of a half: an exponent of all ones
                            if (some) {
#pragma unroll
                                for (int c = 0; c < C::HALVES * 8; ++c) {
                                    const uint4 u = *reinterpret_cast<const uint4 *>(rp + (c >> 3) * C::BOX + (((c & 7) ^ (r & 7)) << 4));
                                    big |= ((u.x & 0x7fff7fffu) + 0x00800080u) | ((u.y & 0x7fff7fffu) + 0x00800080u) |
                                           ((u.z & 0x7fff7fffu) + 0x00800080u) | ((u.w & 0x7fff7fffu) + 0x00800080u);
                                }
                            }
                            const bool inf = (big & 0x80008000u) != 0;
                            if (!live) {
#pragma unroll
                                for (int c = 0; c < C::HALVES * 8; ++c)
                                    *reinterpret_cast<uint4 *>(rp + (c >> 3) * C::BOX + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                            } else if (inf) {
#pragma unroll 1
                                for (int c = 0; c < C::HALVES * 8; ++c) {
                                    uint4 *u = reinterpret_cast<uint4 *>(rp + (c >> 3) * C::BOX + (((c & 7) ^ (r & 7)) << 4));
                                    *u = finite(*u);
                                }
                            }
                            word = __ballot_sync(0xffffffffu, inf);
                        }
                        if (lane == 0) s_poison[(pos % kPoisonRing) * 4 + g] = word;
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_full + st);
                }
            }
        }
        if (!p.tree && blockIdx.x == 0) check_ranges(p.q_start, p.B, p.N, p.status);
        __syncwarp();
    } else if (warp == kWarpMma) {
        // -------------------------------------------------------------- MMA
        regs_dec<C::REGS_OTHER>();
        const uint64_t qdesc = smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
        const uint64_t kdesc = smem_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
        const uint64_t vdesc = smem_desc_sw128(smem_u32(smem + C::OFF_V), C::BOX, 1024);
        int kst = 0, kph = 0, vst = 0, vph = 0;     // ring places of the next K / V tile
        int cnt0 = 0, cnt1 = 0;                     // softmax steps of each group so far
        int items = 0;
        bool ok = true;
        w.start(p, s_start);
        while (ok && w.next(p)) {
            const int two = ONE ? 0 : w.it.two, n_steps = (w.j1 - w.j0) << two;
            int kw = 0;                             // K tiles of the item waited for
            auto qk = [&](int s) -> bool {          // scores of step s
                const int g = s & 1, tile = s >> two;
                if (tile >= kw) {
                    if (!warp_wait(k_full + kst, kph)) return false;
                    ++kw;
                    tc_fence_after();
                }
                const uint64_t kd = kdesc + ((kst * C::TILE) >> 4);
                const uint64_t qd = qdesc + (two ? (g * C::TILE) >> 4 : 0);
                const bool done = !two || g == 1;   // the tile's last use
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * C::BOX + (kk & 3) * 32) >> 4;
                        mma_ss(tmem + C::COL_S + g * 128, qd + off, kd + off, C::IDESC_QK, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(s_full + g);
                    if (done) mma_commit(k_empty + kst);
                    if (s == n_steps - 1) mma_commit(q_empty);
                }
                if (done && ++kst == C::NK) { kst = 0; kph ^= 1; }
                return true;
            };
            ok = warp_wait(q_full, items);
            tc_fence_after();
            for (int s = 0; ok && s < min(2, n_steps); ++s) ok = qk(s);
            if (ok) ok = warp_wait(o_empty, items + 1);
            for (int s = 0; ok && s < n_steps; ++s) {
                const int g = s & 1;
                if (!two || g == 0) {
                    ok = warp_wait(v_full + vst, vph);
                }
                const uint64_t vd = vdesc + ((vst * C::TILE) >> 4);
                const bool done = !two || g == 1;
                auto pv = [&](int kk) {
                    mma_ts(tmem + C::COL_O + g * D, tmem + C::COL_S + g * 128 + 64 + kk * 8, vd + ((kk * 16 * 128) >> 4), C::IDESC_PV,
                           (s > 1 || kk != 4) ? 1u : 0u);
                };
                // the upper 64 keys while the softmax group works on the lower ones
                if (ok) ok = warp_wait(p_ready + 2 * g, g ? cnt1 : cnt0);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 4; kk < 8; ++kk) pv(kk);
                }
                ok = warp_wait(p_ready + 2 * g + 1, g ? cnt1 : cnt0);
                if (!ok) break;
                if (g) ++cnt1; else ++cnt0;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) pv(kk);
                    if (done) mma_commit(v_empty + vst);
                    if (s == n_steps - 1) mma_commit(o_full);
                }
                if (done && ++vst == C::NV) { vst = 0; vph ^= 1; }
                if (s + 2 < n_steps) ok = qk(s + 2);
            }
            ++items;
        }
        if (elect_one()) mma_commit(drain);         // all MMAs issued are done before TMEM is freed
        warp_wait(drain, 0);
    } else if (warp >= kWarpLoad) {
        // ------------- loaders (e4m3 cache): four warps for K, four for V
        if constexpr (Q8) {
            regs_dec<C::REGS_LOAD>();
            const bool is_v = warp >= kWarpLoad + 4;
            const int lw = (warp - kWarpLoad) & 3, set_bar = is_v ? 3 : 2;
            // A lane converts one row, 8 codes at a time, in an order of its own: piece
            // i ^ turn.  The turns are chosen such that 16 lanes' loads meet 16 different
            // 8-byte banks and 8 lanes' stores 8 different 16-byte ones behind the
            // swizzle (D = 128: r -> 2r in GF(8), for which r and r + 2r are both
            // permutations; D = 64, two rows to 128 bytes: r >> 1).
            const int row = lw * 32 + lane;
            const uint32_t turn = D == 128 ? (((lane << 1) & 6) ^ (lane & 4 ? 3 : 0)) | (lane & 8) : (lane >> 1) & 7;
            const uint32_t raw_off = C::TILE - C::RAW + row * D, out_off = row * 128;
            Walk &lwk = *reinterpret_cast<Walk *>(smem + C::OFF_WALK + (is_v ? 2 : 1) * C::WALK_BYTES);
            volatile int *more = reinterpret_cast<volatile int *>(reinterpret_cast<uint8_t *>(&lwk) + C::WALK_BYTES - 4);
            const bool first_thread = lw == 0 && lane == 0;
            const int ns = is_v ? C::NV : C::NK;
            uint8_t *ring = smem + (is_v ? C::OFF_V : C::OFF_K);
            uint64_t *raw = is_v ? v_raw : k_raw, *full = is_v ? v_full : k_full;
            int st = 0, ph = 0, pos = 0;
            bool ok = true;
            if (first_thread) lwk.start(p, s_start);
            // A stage's codes to f16, in place, times the row's `mult` (0: zeros).  At
            // D = 128 a row's codes lie where its own second half goes, so a lane needs
            // no other's progress; at D = 64 they lie where other warps' rows go.  All
            // loads of the row first: beside the MMAs' traffic a load from shared memory
            // takes hundreds of cycles (four at a time, with the multipliers by shuffles:
            // 2400 cycles a tile against 1100).
            uint2 u[D / 8];
            auto read_row = [&](const uint8_t *stage) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) u[i] = *reinterpret_cast<const uint2 *>(stage + raw_off + ((turn ^ i) << 3));
            };
            auto write_row = [&](uint8_t *stage, uint32_t mult) {
                if (D == 64) bar_sync(set_bar, 128);
                const uint32_t keep = mult ? 0xffffffffu : 0u;      // (NaN codes)
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint2 a = e4m3x4_to_f16x4(u[i].x & keep, mult), b = e4m3x4_to_f16x4(u[i].y & keep, mult);
                    const uint32_t c = turn ^ i;
                    *reinterpret_cast<uint4 *>(stage + (c >> 3) * C::BOX + out_off + (((c & 7) ^ (row & 7)) << 4)) =
                        make_uint4(a.x, a.y, b.x, b.y);
                }
            };
            // largest scale byte of the live rows [a, z) (NaN rows aside), with kEach where
            // the least lies more than `spread` below it; w4: bytes of rows 4 * lane ..
            auto tile_exp = [&](uint32_t w4, int a, int z, int spread) {
                uint32_t most = kScaleMin, least = kScaleNan;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = (w4 >> (8 * i)) & 255, r = 4 * lane + i;
                    if (static_cast<int>(r) >= a && static_cast<int>(r) < z && x != kScaleNan) {
                        most = max(most, x);
                        least = min(least, x);
                    }
                }
                most = __reduce_max_sync(0xffffffffu, most);
                least = __reduce_min_sync(0xffffffffu, least);
                return static_cast<int>(most) | (most > least + spread ? kEach : 0);
            };
            const int spread = is_v ? kSpreadV : kSpreadK;
            for (;;) {
                bar_sync(set_bar, 128);
                if (first_thread) *more = lwk.next(p);
                bar_sync(set_bar, 128);
                if (!*more) break;
                const int j0 = lwk.j0, j1 = lwk.j1, cache_tiles = lwk.it.cache_tiles;
                const int lo = lwk.it.lo, hi = lwk.it.hi, base = lwk.it.base;
                for (int j = j0; j < j1; ++j, ++pos) {
                    uint8_t *stage = ring + st * C::TILE;
                    if (ok) ok = warp_wait(raw + st, ph);
                    const int at = pos % kPoisonRing;
                    uint32_t *word = s_poison + at * 4 + lw;
                    if (j < cache_tiles) {
                        const int a = lo - (base + j * 128), z = hi - (base + j * 128);
                        const bool live = row >= a && row < z;
                        const uint8_t *sc = is_v ? smem + C::OFF_SCALE_V + st * 128 : s_scale + at * 256;
                        const uint8_t *scv = is_v ? sc : sc + 128;
                        const int e = sc[row], ev = scv[row];
                        const int E = tile_exp(*reinterpret_cast<const uint32_t *>(sc + 4 * lane), a, z, spread);
                        if (!is_v) {
                            // V rows held as NaN, and V's E, are told to the softmax groups with K
                            const uint32_t nan = __ballot_sync(0xffffffffu, live && ev == kScaleNan);
                            const int Ev = tile_exp(*reinterpret_cast<const uint32_t *>(scv + 4 * lane), a, z, kSpreadV);
                            if (lane == 0) *word = nan;
                            if (first_thread) s_exp[at] = make_int2(E, Ev);
                        }
                        read_row(stage);
                        write_row(stage, !live ? 0u : e != kScaleNan ? f16_pow2(E & kEach ? 0 : e - E) : is_v ? 0u : 0x7e007e00u);
                    } else {
                        // tree rows (bf16), one a lane, scaled into f16 by the tile's largest value or,
                        // where the rows' largest values lie far apart, by their own (2^(127 - e);
                        // rows of zeros are zeros under any).  Rows behind the tree are zeroed, and so
                        // are a V row's infinities and NaN, and the softmax groups told (they wait for
                        // this tile).
                        const int r = lw * 32 + lane, live = min(128, p.N - (j - cache_tiles) * 128);
                        uint8_t *rp = stage + r * 128;
                        auto piece = [&](int x) { return reinterpret_cast<uint4 *>(rp + (x >> 3) * C::BOX + (((x & 7) ^ (r & 7)) << 4)); };
                        uint32_t big = 0;
#pragma unroll 4
                        for (int x = 0; x < D / 8; ++x) big = max_bits(*piece(x), big);
                        big = halves_max(big);
                        const bool inf = big >= 0x7f80u;
                        if (inf) {                          // (the scale is that of the numbers)
                            big = 0;
#pragma unroll 1
                            for (int x = 0; x < D / 8; ++x) {
                                if (is_v) *piece(x) = finite(*piece(x));
                                big = max_bits(finite(*piece(x)), big);
                            }
                            big = halves_max(big);
                        }
                        uint32_t *red = reinterpret_cast<uint32_t *>(smem + C::OFF_RED) + (is_v ? 4 : 0);
                        const int e = 127 - f16_shift(big, 112);        // 15 .. 240
                        const bool counts = r < live && big != 0;
                        const uint32_t most = __reduce_max_sync(0xffffffffu, counts ? e : 15);
                        const uint32_t least = __reduce_min_sync(0xffffffffu, counts ? e : 255);
                        bar_sync(set_bar, 128);
                        if (lane == 0) red[lw] = most | (least << 16);
                        bar_sync(set_bar, 128);
                        int E = 15, lowest = 255;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            E = max(E, static_cast<int>(red[i] & 0xffffu));
                            lowest = min(lowest, static_cast<int>(red[i] >> 16));
                        }
                        const bool each = E > lowest + spread;
                        const float mul = pow2(127 - (each ? e : E));
#pragma unroll 4
                        for (int x = 0; x < D / 8; ++x) *piece(x) = r >= live ? make_uint4(0u, 0u, 0u, 0u) : to_f16(*piece(x), mul);
                        s_scale[at * 256 + (is_v ? 128 : 0) + r] = static_cast<uint8_t>(e);
                        if (is_v) {
                            const uint32_t nan = __ballot_sync(0xffffffffu, r < live && inf);
                            if (lane == 0) *word = nan;
                        }
                        if (first_thread) (is_v ? s_exp[at].y : s_exp[at].x) = E | (each ? kEach : 0);
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full + st);
                    if (++st == ns) { st = 0; ph ^= 1; }
                }
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- softmax
        regs_inc<C::REGS_SOFTMAX>();
        const int grp = (warp - kWarpSoftmax) >> 2, wq = warp & 3;
        const int r = wq * 32 + lane;                       // row of the tile = TMEM lane
        const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t t_s = tmem + lane_addr + C::COL_S + grp * 128;
        const uint32_t t_o = tmem + lane_addr + C::COL_O;
        const float nan = __int_as_float(0x7fc00000);
        int cnt = 0, items = 0, pos = 0;                    // steps of this group, items, key tiles so far
        bool ok = true;
        // One walk for both groups, in shared memory: its thirty values would
        // cost every softmax thread as many registers.
        static_assert(sizeof(Walk) + 4 <= C::WALK_BYTES, "shared memory of the walk");
        Walk &w = *reinterpret_cast<Walk *>(smem + C::OFF_WALK);
        volatile int *more = reinterpret_cast<volatile int *>(smem + C::OFF_WALK + C::WALK_BYTES - 4);
        const bool first_thread = threadIdx.x == kWarpSoftmax * 32;
        if (first_thread) w.start(p, s_start);
        // both partial slots' headers are written by every launch
        int head_first = -1, head_last = -1;
        for (;;) {
            if (first_thread) *more = w.next(p);
            bar_sync(1, 256);
            if (!*more) break;
            const int two = ONE ? 0 : w.it.two;
            const int row = two ? grp * 128 + r : r;        // row of the item
            const bool valid = row < w.it.rows;
            const bool warp_active = (two ? grp * 128 : 0) + wq * 32 < w.it.rows;
            const int pr = w.it.r0 + (valid ? row : 0);     // packed row
            int t = 0, g = 0;
            size_t orow;
            const __nv_bfloat16 *qp;
            if (p.tree) {
                t = pr % p.N;
                orow = (static_cast<size_t>(w.cur_b) * p.Hq + static_cast<size_t>(w.cur_kvh) * p.G) * p.N + pr;
                qp = p.q + orow * D;
            } else {
                t = div_g(p, pr);
                g = pr - t * p.G;
                const int h = w.cur_kvh * p.G + g;
                orow = static_cast<size_t>(w.s.s0 + t) * p.Hq + h;
                qp = p.q + (w.s.s0 + t) * p.q_stride + static_cast<size_t>(h) * D;
            }
            if (w.s.bad && first_thread) raise_status(p.status, kStatusPrefixLenRange);
            bool row_nan = w.s.bad, row_inf = false;        // row_inf: sees a V row that lost some
            float c2_row = p.scale_log2;
            // ---- Q into shared memory (one row tile: each group half of the columns)
            {
                // The warp's 32 rows, a row's pieces on neighbouring lanes: a load per row
                // and thread touched 32 lines each time, 4 us an item.
                const int ch0 = two ? 0 : grp * (D / 16), nch = two ? D / 8 : D / 16;
                const int cs = Q8 || two ? (D == 128 ? 4 : 3) : (D == 128 ? 3 : 2);   // log2 of the pieces read of a row
                const int rpi = 32 >> cs, ch = (Q8 ? 0 : ch0) + (lane & ((1 << cs) - 1));
                const uint32_t rows = __ballot_sync(0xffffffffu, valid);
                const unsigned long long q_at = reinterpret_cast<unsigned long long>(qp);
                if (ok) ok = warp_wait(q_empty, items + 1);
                uint8_t *qs = smem + C::OFF_Q + (two ? grp * C::TILE : 0) + wq * 32 * 128;
                for (int i0 = 0; i0 < (1 << cs); i0 += 4) {
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = (i0 + i) * rpi + (lane >> cs);
                        const uint4 *src = reinterpret_cast<const uint4 *>(__shfl_sync(0xffffffffu, q_at, rr));
                        v[i] = (rows >> rr) & 1u ? src[ch] : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = (i0 + i) * rpi + (lane >> cs);
                        uint4 y = v[i];
                        if constexpr (Q8) {             // (the shift takes the whole row's largest value)
                            uint32_t big = halves_max(max_bits(v[i], 0u));
                            for (int o = 1; o < (1 << cs); o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
                            const int up = f16_shift(big, 100);
                            const int mine = __shfl_sync(0xffffffffu, up, (lane & (rpi - 1)) << cs);
                            if (lane / rpi == i0 + i) c2_row = p.scale_log2 * pow2(-mine);
                            y = to_f16(v[i], pow2(up));
                        }
                        if (ch >= ch0 && ch < ch0 + nch)
                            *reinterpret_cast<uint4 *>(qs + (ch >> 3) * C::BOX + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = y;
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            bool tree_bad = false;
            if (w.j1 > w.it.cache_tiles) {                  // this CTA has keys of the tree
                const int i = (warp - kWarpSoftmax) * 32 + lane;
                bool bad = false;
                if (i < p.N) {
                    const int up = p.parent[static_cast<size_t>(w.cur_b) * p.N + i];
                    bad = up < -1 || up >= i;
                    s_parent[i] = static_cast<uint8_t>(up + 1);
                }
                __syncwarp();
                tree_bad = bar_or(1, 256, bad);
                if (tree_bad && i == 0) raise_status(p.status, kStatusBadParent);
                row_nan |= tree_bad;
            }
            const int row_hi = p.tree ? w.it.hi : (w.s.bad ? 0 : w.s.L + t + 1);
            const int row_lo = p.window > 0 ? max(0, row_hi - p.window) : 0;

            const int it_base = w.it.base, it_all_lo = w.it.all_lo, it_all_hi = w.it.all_hi, it_cache_tiles = w.it.cache_tiles;
            float m_run = -INFINITY;
            float e_run = 0.f;                              // (e4m3) O is in units of 2^(m_run + e_run - 127)
            uint64_t l2 = 0, r2 = 0;                        // sums of 2^(x - m_run); (bf16) of what P holds of them
            const int j0 = w.j0, n_tiles = w.j1 - j0;
            const int step = two ? 1 : 2;
            for (int jj = two ? 0 : grp; jj < n_tiles; jj += step) {
                const int j = j0 + jj;
                if (ok) ok = warp_wait(s_full + grp, cnt);
                ++cnt;
                tc_fence_after();
                if (ok && warp_active) {
                    // the keys of a partly visible tile that this row sees
                    const bool of_tree = j >= it_cache_tiles;
                    const int key0 = it_base + j * 128;
                    const bool masked = of_tree || key0 < it_all_lo || key0 + 128 > it_all_hi;
                    uint32_t see[4];
                    uint4 bad_v = make_uint4(0u, 0u, 0u, 0u);
                    if (Q8 && !of_tree) bad_v = *reinterpret_cast<const uint4 *>(s_poison + ((pos + jj) % kPoisonRing) * 4);
                    if (masked) {
                        if (of_tree) {
                            const int first = (j - it_cache_tiles) * 128;
#pragma unroll
                            for (int i = 0; i < 4; ++i) see[i] = 0;
                            // (parents lie below their nodes, so the walk ends)
                            for (int node = tree_bad ? -1 : t; node >= 0; node = s_parent[node] - 1) {
                                const int d = node - first;
#pragma unroll
                                for (int i = 0; i < 4; ++i) see[i] |= (d >> 5) == i ? 1u << (d & 31) : 0u;
                            }
                        } else {
                            const int a = row_lo - key0, z = row_hi - key0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) see[i] = bit_range(a - 32 * i, z - 32 * i);
                        }
                        if (!Q8 || of_tree) {           // the fixer's or the loaders' word on this tile
                            __syncwarp();
                            ok = warp_wait(v_full + (pos + jj) % C::NV, (pos + jj) / C::NV);
                            bad_v = *reinterpret_cast<const uint4 *>(s_poison + ((pos + jj) % kPoisonRing) * 4);
                        }
                        if ((see[0] & bad_v.x) | (see[1] & bad_v.y) | (see[2] & bad_v.z) | (see[3] & bad_v.w))
                            (Q8 && !of_tree ? row_nan : row_inf) = true;
                        __syncwarp();
                    } else if (Q8) {
                        if (bad_v.x | bad_v.y | bad_v.z | bad_v.w) row_nan = true;
                    }
                    float c2 = c2_row;
                    bool resc = false;
                    float alpha = 1.f, shift = 0.f;         // P is 2^(x - m + shift)
                    // Passes over the row's 128 scores, 32 at a time, from tensor memory each
                    // time: hidden keys to -inf (partly visible tiles), the maximum, the
                    // weights.  One pass with all 128 in registers took the same time (983
                    // against 990 us for the prefill) and left the e4m3 loaders too few.
                    if (masked) {
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            uint32_t x[32];
                            tmem_ld32(t_s + 32 * q, x);
                            tmem_wait_ld();
                            const uint32_t bits = q == 0 ? see[0] : q == 1 ? see[1] : q == 2 ? see[2] : see[3];
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = (bits >> i) & 1u ? x[i] : __float_as_uint(-INFINITY);
                            tmem_st32(t_s + 32 * q, x);
                        }
                        tmem_wait_st();
                    }
                    // (e4m3) the scales of the tile's rows, or the codes as they are and each
                    // row's own scale: K's on the scores, V's on the weights
                    bool each_v = false;
                    float e_v = 0.f, top = -INFINITY;       // V's scale; with each_v the largest x + scale
                    const uint8_t *keys = s_scale + ((pos + jj) % kPoisonRing) * 256;
                    if constexpr (Q8) {
                        const int2 E = s_exp[(pos + jj) % kPoisonRing];
                        const bool each_k = (E.x & kEach) != 0;
                        each_v = (E.y & kEach) != 0;
                        e_v = static_cast<float>(E.y & 255);
                        if (each_k || each_v) {
                            if (!each_k) c2 *= pow2((E.x & 255) - 127);
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
                                uint32_t x[16];
                                tmem_ld16(t_s + 16 * q, x);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    float y = __uint_as_float(x[i]);
                                    if (each_k) {           // (a hidden key's byte may be anything)
                                        const float k = c2 * __uint_as_float(static_cast<uint32_t>(keys[16 * q + i]) << 23);
                                        y = y == -INFINITY ? y : y * k;
                                        x[i] = __float_as_uint(y);
                                    } else {
                                        y *= c2;
                                    }
                                    top = fmaxf(top, y + static_cast<float>(keys[128 + 16 * q + i]));
                                }
                                if (each_k) tmem_st16(t_s + 16 * q, x);
                            }
                            if (each_k) {
                                tmem_wait_st();
                                c2 = 1.f;
                            }
                        } else {
                            c2 *= pow2(E.x - 127);
                        }
                    }
                    float mt = -INFINITY;
                    uint32_t x[2][32];                  // two quarters, the next on its way
                    tmem_ld32(t_s, x[0]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        tmem_wait_ld();
                        pin(x[q & 1]);
                        if (q < 3) tmem_ld32(t_s + 32 * (q + 1), x[(q + 1) & 1]);
                        float a = -INFINITY, b2 = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            a = max3(a, __uint_as_float(x[q & 1][i]), __uint_as_float(x[q & 1][i + 1]));
                            b2 = max3(b2, __uint_as_float(x[q & 1][i + 2]), __uint_as_float(x[q & 1][i + 3]));
                        }
                        mt = max3(mt, a, b2);
                    }
                    const float m_tile = mt * c2;
                    if (m_tile != m_tile) row_nan = true;
                    if (!each_v) top = m_tile + e_v;
                    if (m_tile > m_run + 8.f) {
                        const float d = m_run - m_tile, a = ex2(d);   // 0 on the first tile with a visible key
                        l2 = fma2(l2, f2(a, a), 0ull);
                        if constexpr (!Q8) r2 = fma2(r2, f2(a, a), 0ull);
                        alpha = a;
                        resc = jj >= step;                  // (O holds nothing before the group's second tile)
                        m_run = m_tile;
                        if constexpr (Q8) {                 // the reference m_run + e_run stays or grows
                            const float e = fmaxf(rintf(d + e_run), ceilf(top - m_run));
                            alpha = ex2(d + (e_run - e));
                            e_run = e;
                        }
                    } else if (Q8 && top > m_run + e_run + 8.f) {
                        const float e = ceilf(top - m_run);
                        alpha = ex2(e_run - e);
                        resc = jj >= step;
                        e_run = e;
                    }
                    if constexpr (Q8) shift = each_v ? 0.f : fmaxf(e_v - e_run, -60.f);   // (2^-52 is 0 in f16)
                    if (__any_sync(0xffffffffu, resc)) {
                        // this tile's scores were committed after P*V of the group's previous
                        // tile, so O[grp] is complete, and P*V of this tile waits for this warp
                        const float a = resc ? alpha : 1.f;
#pragma unroll 1
                        for (int col = 0; col < D; col += 32) {
                            uint32_t ro[32];
                            tmem_ld32(t_o + grp * D + col, ro);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) ro[i] = __float_as_uint(__uint_as_float(ro[i]) * a);
                            tmem_st32(t_o + grp * D + col, ro);
                        }
                    }
                    const float mu = (m_run == -INFINITY ? 0.f : m_run) - shift;
                    const uint64_t cc = f2(c2, c2), nm = f2(-mu, -mu);
                    uint64_t lt = 0;
                    // (All exponentials on the exp2 unit: a polynomial on the FMA pipe for one
                    // in 2, 4, 5 or 8 of them was 1 to 4 % slower for the prefill.)
                    // From the last quarter to the first (bf16: the last two are in registers
                    // still): P of quarter q on the columns 64 + 16q .., whose scores have
                    // been read by then.
                    auto weights = [&](const uint32_t (&y)[32], int q) {
                        uint32_t pk[16];
                        uint64_t ls[2] = {0ull, 0ull}, rs[2] = {0ull, 0ull};
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const uint64_t x2 = fma2(f2(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), cc, nm);
                            const float2 z = unf2(x2), e = make_float2(ex2(z.x), ex2(z.y));
                            pk[k] = Q8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
                            ls[k & 1] = add2(ls[k & 1], f2(e.x, e.y));
                            if constexpr (!Q8) rs[k & 1] = add2(rs[k & 1], f2(bf16_lo(pk[k]), bf16_hi(pk[k])));
                        }
                        lt = add2(lt, add2(ls[0], ls[1]));
                        if constexpr (!Q8) r2 = add2(r2, add2(rs[0], rs[1]));
                        tmem_st16(t_s + 64 + 16 * q, pk);
                    };
                    auto half_done = [&]() {
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_ready + 2 * grp);
                    };
                    if constexpr (!Q8) {
                        weights(x[1], 3);
                        tmem_ld32(t_s + 32, x[1]);
                        weights(x[0], 2);
                        tmem_ld32(t_s, x[0]);
                        half_done();
                        tmem_wait_ld();
                        pin(x[1]);
                        pin(x[0]);
                        weights(x[1], 1);
                        weights(x[0], 0);
                    } else if (!each_v) {               // (as a loop: fewer registers)
#pragma unroll 1
                        for (int q = 3; q >= 0; --q) {
                            uint32_t y[32];
                            tmem_ld32(t_s + 32 * q, y);
                            tmem_wait_ld();
                            pin(y);
                            weights(y, q);
                            if (q == 2) half_done();
                        }
                    } else {
                        // (w 2^(127 - e_run)) 2^(e - 127): neither leaves fp32's range upwards, e and
                        // e_run being 15 at least; what underflows is 0 in f16.  (255, a NaN row or
                        // one nobody sees: a number for the weight of 0 to meet.)
                        const float unit = ex2(127.f - e_run);
                        const uint64_t uu = f2(unit, unit);
#pragma unroll 1
                        for (int q = 3; q >= 0; --q) {
                            uint32_t y[32];
                            tmem_ld32(t_s + 32 * q, y);
                            tmem_wait_ld();
                            const uint8_t *e = keys + 128 + 32 * q;
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float2 z = unf2(fma2(f2(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), cc, nm));
                                const uint64_t w = f2(ex2(z.x), ex2(z.y));
                                lt = add2(lt, w);
                                const float2 u = unf2(fma2(w, uu, 0ull));
                                y[k] = pack_f16x2(u.x * __uint_as_float(min(static_cast<uint32_t>(e[2 * k]), 254u) << 23),
                                                  u.y * __uint_as_float(min(static_cast<uint32_t>(e[2 * k + 1]), 254u) << 23));
                            }
                            tmem_st16(t_s + 64 + 16 * q, y);
                            if (q == 2) half_done();
                        }
                    }
                    tmem_wait_st();
                    if constexpr (Q8) {
                        const float back = ex2(-shift);
                        l2 = fma2(lt, f2(back, back), l2);
                    } else {
                        l2 = add2(l2, lt);
                    }
                } else if (lane == 0) {
                    mbar_arrive(p_ready + 2 * grp);     // (no rows in this warp, or the CTA gave up)
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 2 * grp + 1);
            }

            // ------------------------------------------------------ epilogue
            if (ok) ok = warp_wait(o_full, items);
            tc_fence_after();
            const float2 lp = unf2(l2), rp = unf2(r2);
            float l = m_run == -INFINITY ? 0.f : lp.x + lp.y, m = m_run;
            float div = Q8 || m_run == -INFINITY ? l : rp.x + rp.y;   // what O is divided by
            float a0 = 1.f, a1 = 0.f;
            float o0 = Q8 ? ex2(e_run - 127.f) : 1.f, o1 = 1.f;      // scales of O[0], O[1] (two row tiles: of the own)
            bool has1 = false;
            if (!two) {                                     // join the groups: key tiles 0, 2, .. and 1, 3, ..
                float *xch = reinterpret_cast<float *>(smem + C::OFF_XCH);
                xch[(grp * 3 + 0) * 128 + r] = m;
                xch[(grp * 3 + 1) * 128 + r] = row_nan || !ok ? nan : l;   // (a bad row of either group: through the sum)
                xch[(grp * 3 + 2) * 128 + r] = Q8 ? o0 : div;
                xch[(6 + grp) * 128 + r] = row_inf ? 1.f : 0.f;
                bar_sync(1, 256);
                const float m0 = xch[r], m1 = xch[3 * 128 + r];
                m = fmaxf(m0, m1);
                a0 = m0 == -INFINITY ? 0.f : ex2(m0 - m);
                a1 = m1 == -INFINITY ? 0.f : ex2(m1 - m);
                const float l0 = xch[128 + r], l1 = xch[4 * 128 + r];
                l = a0 * l0 + a1 * l1;
                if constexpr (Q8) {
                    o0 = xch[2 * 128 + r];
                    o1 = xch[5 * 128 + r];
                    div = l;
                } else {
                    div = a0 * xch[2 * 128 + r] + a1 * xch[5 * 128 + r];
                }
                row_nan = l0 != l0 || l1 != l1;
                row_inf = xch[6 * 128 + r] + xch[7 * 128 + r] > 0.f;
                has1 = n_tiles > 1;
                if constexpr (!Q8) bar_sync(1, 256);    // (rows are staged there next)
            } else if (!ok) {
                row_nan = true;
            }
            const bool whole = w.j0 == 0 && w.j1 == w.it.nt;
            if (l != l) row_nan = true;
            const float inv = row_nan ? nan : l > 0.f ? 1.f / div : 0.f;
            const float lse = row_nan ? nan : l > 0.f ? (m + lg2(l)) * kLn2 : -INFINITY;
            const int which = w.j0 > 0 ? 0 : 1;             // the CTA's first item, begun elsewhere, or its last
            const long long prow = slot_row(p, blockIdx.x, which) + row;
            const int col0 = two ? 0 : grp * (D / 2), col1 = two ? D : col0 + D / 2;
            if (warp_active) {
                // W columns at a time.  bf16 caches: the rows leave by way of shared memory
                // (Q's, which has been read), so that a store covers whole pieces of few rows
                // (two chunks of 500 tokens 41.6 -> 37.9 us against a row per thread); the
                // trees over e4m3 caches lose 2-3 % by it and store a row per thread.
                constexpr int W = Q8 || C::OFF_K >= 32768 ? 32 : 16;
                static_assert(Q8 || 8 * 32 * W * 4 <= C::OFF_K, "a piece of W columns per warp");
                const float f0 = a0 * inv * o0, f1 = a1 * inv * o1;
                const uint32_t to0 = t_o + (two ? grp * D : 0), to1 = t_o + D;
                uint8_t *buf = smem + C::OFF_Q + (warp - kWarpSoftmax) * 32 * W * 4;
                const uint32_t rows = __ballot_sync(0xffffffffu, valid);
                const int my_row = whole ? static_cast<int>(orow) : row;    // (2^31 rows of out would be 256 GB)
                // the Q 16-byte pieces of each lane's row, piece(i) the i-th: to dst + row * row_bytes
                auto store = [&](auto pieces, auto piece, uint8_t *dst, int row_bytes) {
                    constexpr int Q = decltype(pieces)::value;
                    if constexpr (Q8) {
                        if (valid) {
#pragma unroll
                            for (int i = 0; i < Q; ++i)
                                *reinterpret_cast<uint4 *>(dst + static_cast<long long>(my_row) * row_bytes + i * 16) = piece(i);
                        }
                        __syncwarp();
                    } else {
                        // piece i of a row at i XOR the row's place among those that share 128 bytes
                        auto at = [&](int rr, int i) { return reinterpret_cast<uint4 *>(buf) + rr * Q + (i ^ (rr * Q / 8 & (Q - 1))); };
#pragma unroll
                        for (int i = 0; i < Q; ++i) *at(lane, i) = piece(i);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < Q; ++i) {
                            const int rr = (i * 32 + lane) / Q, q = lane % Q;
                            const long long to = __shfl_sync(0xffffffffu, my_row, rr);
                            const uint4 v = *at(rr, q);
                            if ((rows >> rr) & 1u) *reinterpret_cast<uint4 *>(dst + to * row_bytes + q * 16) = v;
                        }
                        __syncwarp();
                    }
                };
#pragma unroll 1
                for (int col = col0; col < col1; col += W) {
                    uint32_t x0[W], x1[W];
                    float y[W];
                    if constexpr (W == 32) {
                        tmem_ld32(to0 + col, x0);
                        if (has1) tmem_ld32(to1 + col, x1);
                    } else {
                        tmem_ld16(to0 + col, x0);
                        if (has1) tmem_ld16(to1 + col, x1);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        y[i] = __uint_as_float(x0[i]) * f0;
                        if (has1) y[i] = fmaf(__uint_as_float(x1[i]), f1, y[i]);
                        if (l == 0.f && !row_nan) y[i] = 0.f;
                    }
                    if (whole)
                        store(Int<W / 8>(), [&](int i) {
                            return make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                              pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
                        }, reinterpret_cast<uint8_t *>(p.out) + col * 2, D * 2);
                    else
                        store(Int<W / 4>(), [&](int i) {
                            return make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]),
                                              __float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3]));
                        }, reinterpret_cast<uint8_t *>(p.o_part + slot_row(p, blockIdx.x, which) * D + col), D * 4);
                }
                if (row_inf && !row_nan && valid) {         // infinities and NaN to their columns
                    auto add_bad = [&](const __nv_bfloat16 *v) {
#pragma unroll 1
                        for (int c = col0; c < col1; ++c) {
                            const float x = __bfloat162float(v[c]);
                            if (fabsf(x) <= 3.4e38f) continue;
                            if (whole) p.out[orow * D + c] = __float2bfloat16(__bfloat162float(p.out[orow * D + c]) + x);
                            else p.o_part[prow * D + c] += x;
                        }
                    };
                    if constexpr (Q8) {
                        const __nv_bfloat16 *v = p.v_tree + (static_cast<size_t>(w.cur_b) * p.Hkv + w.cur_kvh) * p.N * D;
                        for (int node = t; node >= 0; node = s_parent[node] - 1)
                            if (it_cache_tiles + (node >> 7) >= j0 && it_cache_tiles + (node >> 7) < w.j1)
                                add_bad(v + static_cast<size_t>(node) * D);
                    } else {
                        const int32_t *table = p.cache.block_table + static_cast<size_t>(w.cur_b) * p.cache.max_blocks;
                        for (int j = j0; j < w.j1; ++j) {
                            if (!w.partial(j)) continue;
                            for (int key = max(row_lo, w.key0(j)); key < min(row_hi, w.key0(j) + 128); ++key) {
                                int n = table[key >> bsh];
                                if (n < 0 || n >= p.cache.num_blocks) n = 0;    // (as the producers)
                                const size_t at = (static_cast<size_t>(n) * p.Hkv + w.cur_kvh) * bs + (key & (bs - 1));
                                add_bad(static_cast<const __nv_bfloat16 *>(p.cache.v) + at * D);
                            }
                        }
                    }
                }
                if (valid && (two || grp == 0)) {
                    if (whole) p.lse[orow] = lse;
                    else p.lse_part[prow] = lse;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty);
            if (!whole && first_thread) {
                write_head(p, w, s_start, which);
                if (which == 0) head_first = 1; else head_last = 1;
            }
            ++items;
            pos += n_tiles;
            bar_sync(1, 256);       // the item's fields, parents and exchanged sums are read; the next may come
        }
        if (first_thread) {
            if (head_first < 0) p.heads[2 * blockIdx.x].rows = 0;
            if (head_last < 0) p.heads[2 * blockIdx.x + 1].rows = 0;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// -------------------------------------------------------------------- merge
// Rows of items that crossed CTA borders: the partials of an item are slot 1
// of the CTA it begins in and slots 0 of the next n - 1.  One warp per row:
//   out = sum_c e^{lse_c - M} o_c / sum_c e^{lse_c - M},  lse = M + ln(sum).
// Bound by latency: the header, then rounds of loads.  Few rows were split over
// many CTAs (decode: eight segments at a time), many rows over two or three
// (two segments of four rows at a time).
template <int D, int R, int U>       // R rows of a warp and U segments at a time
__global__ void __launch_bounds__(256)
chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int DPL = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, cta = blockIdx.x;
    const PartHead hd = p.heads[2 * cta + 1];
    const int n = min(hd.n, p.grid - cta);
    const float nan = __int_as_float(0x7fc00000);
    for (int row0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * R; row0 < hd.rows; row0 += gridDim.y * 8 * R) {
        auto slot = [&](int i, int r) { return slot_row(p, cta + i, i == 0 ? 1 : 0) + min(row0 + r, hd.rows - 1); };
        // one pass over the segments with running maxima
        float m[R], sum[R], acc[R][DPL];
        bool bad[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            sum[r] = 0.f;
            bad[r] = false;
#pragma unroll
            for (int k = 0; k < DPL; ++k) acc[r][k] = 0.f;
        }
        for (int i0 = 0; i0 < n; i0 += U) {
            float ls[U][R], v[U][R][DPL];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const long long at = slot(min(i0 + u, n - 1), r);
                    ls[u][r] = p.lse_part[at];
                    const float *src = p.o_part + at * D + lane * DPL;
                    if constexpr (DPL == 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(src);
                        v[u][r][0] = x.x; v[u][r][1] = x.y; v[u][r][2] = x.z; v[u][r][3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2 *>(src);
                        v[u][r][0] = x.x; v[u][r][1] = x.y;
                    }
                }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mn = m[r];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    bad[r] |= ls[u][r] != ls[u][r];
                    if (i0 + u >= n) ls[u][r] = -INFINITY;
                    mn = fmaxf(mn, ls[u][r]);
                }
                if (mn == -INFINITY) continue;          // (no visible key so far)
                const float a = ex2((m[r] - mn) * kLog2e);
                m[r] = mn;
                sum[r] *= a;
#pragma unroll
                for (int k = 0; k < DPL; ++k) acc[r][k] *= a;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (ls[u][r] == -INFINITY) continue;    // (a segment without visible keys, or none)
                    const float w = ex2((ls[u][r] - mn) * kLog2e);
                    sum[r] += w;
#pragma unroll
                    for (int k = 0; k < DPL; ++k) acc[r][k] = fmaf(w, v[u][r][k], acc[r][k]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= hd.rows) break;
            const float inv = bad[r] ? nan : sum[r] > 0.f ? 1.f / sum[r] : 0.f;
            const float lse = bad[r] ? nan : sum[r] > 0.f ? m[r] + lg2(sum[r]) * kLn2 : -INFINITY;
            const int pr = hd.r0 + row0 + r;
            size_t orow;
            if (p.tree) {
                orow = (static_cast<size_t>(hd.b) * p.Hq + static_cast<size_t>(hd.kvh) * p.G) * p.N + pr;
            } else {
                const int t = div_g(p, pr);
                orow = static_cast<size_t>(hd.s0 + t) * p.Hq + hd.kvh * p.G + (pr - t * p.G);
            }
            __nv_bfloat16 *dst = p.out + orow * D + lane * DPL;
            if constexpr (DPL == 4) {
                uint2 pk;
                pk.x = pack_bf16x2(acc[r][0] * inv, acc[r][1] * inv);
                pk.y = pack_bf16x2(acc[r][2] * inv, acc[r][3] * inv);
                *reinterpret_cast<uint2 *>(dst) = pk;
            } else {
                *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(acc[r][0] * inv, acc[r][1] * inv);
            }
            if (lane == 0) p.lse[orow] = lse;
        }
    }
}

cudaError_t launch_chunk_merge(const ChunkParams &p, cudaStream_t stream) {
    if (p.slot_rows <= 16) {
        OverlappedLaunch l(dim3(p.grid, (p.slot_rows + 7) / 8), dim3(256), 0, stream);
        return p.D == 128 ? cudaLaunchKernelEx(&l.cfg, chunk_merge_kernel<128, 1, 8>, p)
                          : cudaLaunchKernelEx(&l.cfg, chunk_merge_kernel<64, 1, 8>, p);
    }
    OverlappedLaunch l(dim3(p.grid, (p.slot_rows + 31) / 32), dim3(256), 0, stream);
    return p.D == 128 ? cudaLaunchKernelEx(&l.cfg, chunk_merge_kernel<128, 4, 2>, p)
                      : cudaLaunchKernelEx(&l.cfg, chunk_merge_kernel<64, 4, 2>, p);
}

namespace {

template <int D, bool Q8, bool ONE>
cudaError_t launch(const ChunkParams &p, const CUtensorMap (&tm)[4], cudaStream_t stream) {
    using C = Cfg<D, Q8, ONE>;
    constexpr int kMaxDev = 64;
    static bool attr_set[kMaxDev] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev || !attr_set[dev]) {
        e = cudaFuncSetAttribute(chunk_tc_kernel<D, Q8, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDev) attr_set[dev] = true;
    }
    OverlappedLaunch l(dim3(p.grid), dim3(C::THREADS), C::SMEM_ALLOC, stream);
    e = cudaLaunchKernelEx(&l.cfg, chunk_tc_kernel<D, Q8, ONE>, tm[0], tm[1], tm[2], tm[3], p);
    if (e != cudaSuccess) return e;
    return launch_chunk_merge(p, stream);
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkParams &p0, const CUtensorMap (&tm)[4], cudaStream_t stream) {
    ChunkParams p = p0;
    // One row tile an item where sequences have at most one on average: deeper
    // rings for what is then bound by the keys' way to the SM.  (8 chunks of 64
    // tokens and 4 heads over 4k keys 66 us against 77 with two; 63 tokens and a chunk
    // of 1900 219 against 238.  Over e4m3 keys the two differ less: 85 against 83,
    // and 318 against 281.)
    const bool one = p.tree ? 1LL * p.N * p.G <= 128 : 1LL * p.N * p.G <= 128LL * p.B;
    p.item_rows = one ? 128 : 256;
    p.slot_rows = p.slot_rows < p.item_rows ? p.slot_rows : p.item_rows;
    // An item's own time (its queries' way in, its rows' way out, the pipeline's
    // fill) is that of about two key tiles of two row tiles, or four of one (ragged
    // windowed chunks: 67 us with a half, 61 with two; measured there only).
    p.c0 = 18;
    p.c1 = 4;
    p.c2 = 8;
    p.min_share = 8;
    const bool q8 = p.cache.k_scale != nullptr;
    if (p.D == 128) {
        if (one) return q8 ? launch<128, true, true>(p, tm, stream) : launch<128, false, true>(p, tm, stream);
        return q8 ? launch<128, true, false>(p, tm, stream) : launch<128, false, false>(p, tm, stream);
    }
    if (one) return q8 ? launch<64, true, true>(p, tm, stream) : launch<64, false, true>(p, tm, stream);
    return q8 ? launch<64, true, false>(p, tm, stream) : launch<64, false, false>(p, tm, stream);
}

}  // namespace hta
