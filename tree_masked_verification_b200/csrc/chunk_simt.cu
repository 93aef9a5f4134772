// chunk_simt.cu -- attention of new tokens to a paged cache on CUDA cores:
// one warp per query row, the row's keys one after the other.
//   o = sum_j e^{x_j - m} v_j / sum_j e^{x_j - m},  x_j = scale * q.k_j,
// over the keys the row sees, with a running max m (the sums are rescaled
// when it moves).
#include "cache_kernels.h"

namespace hta {

namespace {

constexpr int kSimtWarps = 8;

// D/32 values per lane of a cache row
template <int D>
__device__ __forceinline__ void load_cache(const void *cache, const uint8_t *scale, size_t row, int lane, float *x) {
    constexpr int DPL = D / 32;
    if (scale) {
        const uint8_t *c = static_cast<const uint8_t *>(cache) + row * D + lane * DPL;
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < DPL; ++i) w |= static_cast<uint32_t>(c[i]) << (8 * i);
        const uint2 r = dequant_e4m3x4(w, e4m3_mult(scale[row]));
        x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x);
        if constexpr (DPL == 4) { x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y); }
    } else {
        const __nv_bfloat16 *c = static_cast<const __nv_bfloat16 *>(cache) + row * D + lane * DPL;
#pragma unroll
        for (int i = 0; i < DPL; ++i) x[i] = __bfloat162float(c[i]);
    }
}

template <int D>
__global__ void __launch_bounds__(kSimtWarps * 32)
chunk_simt_kernel(const ChunkParams p) {
    constexpr int DPL = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * kSimtWarps + (threadIdx.x >> 5);
    const long long rows = static_cast<long long>(p.tree ? p.B : 1) * p.Hq * p.N;
    if (!p.tree && row == 0) check_ranges(p.q_start, p.B, p.N, p.status);
    if (row >= rows) return;
    int b, h, lo = 0, hi;
    const __nv_bfloat16 *q;
    bool bad;
    if (p.tree) {
        b = static_cast<int>(row / (static_cast<long long>(p.Hq) * p.N));
        h = static_cast<int>(row / p.N % p.Hq);
        q = p.q + row * D;
        hi = p.prefix_len[b];
        bad = hi < 0 || hi > p.L_cap;
    } else {
        const int token = static_cast<int>(row / p.Hq);
        h = static_cast<int>(row % p.Hq);
        q = p.q + token * p.q_stride + static_cast<size_t>(h) * D;
        int s0 = 0, s1 = 0;
        b = find_sequence(p.q_start, p.B, token, s0, s1);
        if (b < 0) return;
        const int L = p.prefix_len[b];
        bad = L < 0 || L > p.L_cap || s1 - s0 > p.L_cap - L;
        hi = bad ? 0 : L + token - s0 + 1;
        if (p.window > 0) lo = max(0, hi - p.window);
    }
    if (bad && lane == 0) raise_status(p.status, kStatusPrefixLenRange);
    float qv[DPL], acc[DPL], m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < DPL; ++i) { qv[i] = __bfloat162float(q[lane * DPL + i]) * p.scale_log2; acc[i] = 0.f; }
    const int kvh = h / p.G, bs = p.cache.block_size;
    for (int j = lo; j < hi && !bad; ++j) {
        int blk = p.cache.block_table[static_cast<size_t>(b) * p.cache.max_blocks + j / bs];
        if (blk < 0 || blk >= p.cache.num_blocks) {
            if (lane == 0) raise_status(p.status, kStatusBadBlock);
            blk = 0;
        }
        const size_t at = (static_cast<size_t>(blk) * p.Hkv + kvh) * bs + j % bs;
        float k[DPL], v[DPL], x = 0.f;
        load_cache<D>(p.cache.k, p.cache.k_scale, at, lane, k);
        load_cache<D>(p.cache.v, p.cache.v_scale, at, lane, v);
#pragma unroll
        for (int i = 0; i < DPL; ++i) x = fmaf(qv[i], k[i], x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        const float mn = fmaxf(m, x);
        const float a = ex2(m - mn), e = ex2(x - mn);
        sum = sum * a + e;
#pragma unroll
        for (int i = 0; i < DPL; ++i) acc[i] = acc[i] * a + e * v[i];
        m = mn;
    }
    const float nan = __int_as_float(0x7fc00000);
    const float inv = bad ? nan : sum > 0.f ? 1.f / sum : 0.f;
    const float lse = bad ? nan : sum > 0.f ? (m + lg2(sum)) * kLn2 : -INFINITY;
    if (p.o_part) {
#pragma unroll
        for (int i = 0; i < DPL; ++i) p.o_part[row * D + lane * DPL + i] = acc[i] * inv;
        if (lane == 0) p.lse_part[row] = lse;
    } else {
#pragma unroll
        for (int i = 0; i < DPL; ++i) p.out[row * D + lane * DPL + i] = __float2bfloat16(acc[i] * inv);
        if (lane == 0) p.lse[row] = lse;
    }
}

}  // namespace

cudaError_t launch_chunk_simt(const ChunkParams &p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.tree ? p.B : 1) * p.Hq * p.N;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>((rows + kSimtWarps - 1) / kSimtWarps));
    cfg.blockDim = dim3(kSimtWarps * 32);
    return p.D == 128 ? cudaLaunchKernelEx(&cfg, chunk_simt_kernel<128>, p)
                      : cudaLaunchKernelEx(&cfg, chunk_simt_kernel<64>, p);
}

}  // namespace hta
