// Dense products for few tokens: a weight-streaming kernel with the operands swapped.
//
// y[t][r] = sum_k W[r][k] x[t][k] for up to N = 128 tokens a CTA: 128 weight rows are the
// MMA's M side and the tokens its N side, so a decode batch of 1 to 16 tokens costs one
// 128 x 16 MMA per K step and every weight byte is read from HBM once.  What bounds it is
// that read.  One CTA streams its rows through a TMA ring (up to 96 KB in flight, two CTAs
// a SM); with few row tiles a cluster of up to 8 CTAs splits K, and its partial sums are
// added through distributed shared memory in rank order (one launch, no workspace, no
// atomics, the same bits every time).
//
//   kSwiglu: rows 0-63 of the tile are gate rows f0..f0+63, rows 64-127 the same up rows;
//            h = silu(g) * u when the partial sums are added.
//   kFp8:    a K-block is one 128-wide scale block; its 128 x N product (exact E4M3
//            products, fp32 sums in tensor memory) is scaled by s_w * s_x[t] and added
//            to fp32 registers.
//   kFp8Store: kFp8 from 16- or 32-bit activations of up to 16 tokens: six warps store the
//            CTA's share of the token rows as E4M3 blocks in shared memory (as
//            fp8_block_quantize does) while the first weights are on their way, so there is
//            no launch before this one and no workspace.
#pragma once

#include "tq_dense.cuh"
#include "tq_fp8_store.cuh"

namespace tq {

constexpr int kSwiglu = 0, kFp8 = 1, kFp8Store = 2;
constexpr int kRowsM = 128;
constexpr int kRowsThreads = 256;   // warp 0 TMA, 1 MMA, 2 TMEM, 4-7 accumulators; all add partial sums

// kFp8Store: the CTA's K-blocks whose stored tokens fit next to the ring, two CTAs a SM.
template <int N>
struct RowsStore {
    static constexpr int kBlockBytes = N * 128 + N * 4;      // E4M3 rows and their scales
    static constexpr int kMost = (46 * 1024) / kBlockBytes;  // 22 for N = 16
};
constexpr int kMostStored = 22;

template <int N, int KIND>
struct RowsShape {
    static constexpr bool kIsFp8 = KIND != kSwiglu;
    static constexpr int kStageBytes = kRowsM * 128 + (KIND == kFp8Store ? 0 : N * 128);
    static constexpr int kMostStages = KIND == kFp8Store ? 4 : 6;
    static constexpr int kStages = (104 * 1024) / kStageBytes < kMostStages ? (104 * 1024) / kStageBytes : kMostStages;
    static constexpr int kAccStages = kIsFp8 ? (N <= 64 ? 4 : 2) : 1;
    static constexpr int kTmemCols = N * kAccStages < 32 ? 32 : N * kAccStages;
    static constexpr int kRing = kStages * kStageBytes;
    static_assert(kStages >= 2 && kRing >= kRowsM * N * 4, "the ring also holds the partial sums");
    static constexpr int kStored = KIND == kFp8Store ? RowsStore<N>::kMost * N * 128 : 0;
    // scales: [acc stage][N] s_x s_w (kFp8), or [K-block][N] s_x (kFp8Store)
    static constexpr int kScales = KIND == kFp8Store ? RowsStore<N>::kMost * N * 4 : KIND == kFp8 ? 4 * kAccStages * N : 0;
    static constexpr int kBytes = kRing + kStored + 1024 + 512 + kScales;
};

struct RowsBars {
    uint64_t full[6], empty[6];
    uint64_t acc_full[4], acc_empty[4];
    uint64_t stored[kMostStored];     // kFp8Store: the K-block's token rows are in shared memory
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(RowsBars) <= 512 && RowsStore<16>::kMost <= kMostStored, "barrier block");

struct RowsArgs {
    int rows;             // tokens
    int width;            // outputs per token: F (kSwiglu) or the weight's rows (kFp8)
    int kblocks;          // K-blocks of 128 bytes
    int out_type;         // tq_dtype
    int accumulate;       // kFp8 with fp32 output: y += ...
    void *out;
    const float *sx;      // [rows][kblocks] (kFp8)
    const void *x;        // [rows][cols] of x_type (kFp8Store)
    int cols, x_type;
    const float *sw;      // [ceil(width / 128)][kblocks]
};

__device__ __forceinline__ void store_out4(void *out, size_t i, const float (&v)[4], int n, int type, bool accumulate) {
    if (type == TQ_DTYPE_F32) {
        float *p = reinterpret_cast<float *>(out) + i;
        if (n == 4 && (i & 3) == 0) {
            float4 w = make_float4(v[0], v[1], v[2], v[3]);
            if (accumulate) {
                const float4 o = *reinterpret_cast<const float4 *>(p);
                w.x += o.x; w.y += o.y; w.z += o.z; w.w += o.w;
            }
            *reinterpret_cast<float4 *>(p) = w;
        } else {
            for (int j = 0; j < n; ++j) p[j] = accumulate ? p[j] + v[j] : v[j];
        }
        return;
    }
    const bool f16 = type == TQ_DTYPE_F16;
    uint16_t *p = reinterpret_cast<uint16_t *>(out) + i;
    const uint32_t a = pack16(v[0], v[1], f16), b = pack16(v[2], v[3], f16);
    if (n == 4 && (i & 3) == 0) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
    } else {
        if (n > 0) p[0] = (uint16_t)(a & 0xFFFFu);
        if (n > 1) p[1] = (uint16_t)(a >> 16);
        if (n > 2) p[2] = (uint16_t)(b & 0xFFFFu);
        if (n > 3) p[3] = (uint16_t)(b >> 16);
    }
}

// Storing warp w of 6: every sixth K-block of the CTA's token rows as E4M3 in the 128-byte
// swizzle the MMA reads, 16 lanes a row and 8 rows in flight.  Rows past the last token are
// left as they are: a product's columns do not mix, and theirs are not stored.
template <typename T, int N>
__device__ __forceinline__ void rows_store(const RowsArgs &args, unsigned char *tokens, float *scales, uint64_t *stored,
                                           int t0, int kb0, int nkb, int w, int lane) {
    const int half = lane >> 4, sub = lane & 15;
    const int rows = min(N, args.rows - t0);
    const T *x = reinterpret_cast<const T *>(args.x) + (size_t)t0 * args.cols;
    for (int i = w; i < nkb; i += 6) {
        const int c = (kb0 + i) * 128 + sub * 8;
        unsigned char *dst = tokens + i * (N * 128);
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 16) {
            float v[8][8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = r0 + 2 * k + half;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][j] = 0.f;
                if (r < rows && c < args.cols) load8<T>(x + (size_t)r * args.cols + c, v[k]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (r0 + 2 * k >= rows) break;
                const int r = r0 + 2 * k + half;
                float scale;
                const uint2 q = fp8_store_block(v[k], scale);
                // 16-byte chunk (sub / 2) of row r lies at chunk (sub / 2) ^ (r mod 8)
                *reinterpret_cast<uint2 *>(dst + r * 128 + (((sub >> 1) ^ (r & 7)) << 4) + (sub & 1) * 8) = q;
                if (sub == 0) scales[i * N + r] = scale;
            }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&stored[i]);
    }
}

template <int N, int KIND>
__global__ void __launch_bounds__(kRowsThreads, KIND != kSwiglu && N > 64 ? 1 : 2)
    dense_rows_kernel(const __grid_constant__ CUtensorMap map_w0, const __grid_constant__ CUtensorMap map_w1,
                      const __grid_constant__ CUtensorMap map_x, const RowsArgs args) {
    using SH = RowsShape<N, KIND>;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    unsigned char *ring = smem_raw + pad;
    unsigned char *tokens = ring + SH::kRing;                            // kFp8Store: [K-block][N][128]
    RowsBars &sm = *reinterpret_cast<RowsBars *>(tokens + SH::kStored);
    float *scales = reinterpret_cast<float *>(tokens + SH::kStored + 512);   // E4M3 only
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    const int tile = blockIdx.x / C;
    const int t0 = blockIdx.y * N;
    const int kb0 = (int)((long long)args.kblocks * rank / C);
    const int nkb = (int)((long long)args.kblocks * (rank + 1) / C) - kb0;
    const int cols_per_kb = SH::kIsFp8 ? 128 : 64;

    if (threadIdx.x == 0) {
        for (int i = 0; i < SH::kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        if (KIND == kFp8Store)
            for (int i = 0; i < RowsStore<N>::kMost; ++i) mbar_init(&sm.stored[i], 1);
        for (int i = 0; i < SH::kAccStages; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], 4);
        }
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc(&sm.tmem_base, SH::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    chain_entry();

    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        if (*(volatile int32_t *)&sm.abort) return false;
        const bool ok = mbar_wait_sleep(bar, parity);
        if (!ok) sm.abort = 1;
        return ok;
    };

    if constexpr (KIND == kFp8Store) {
        // warps 2-7; 4-7 then go on to accumulate
        if (warp >= 2) {
            if (args.x_type == TQ_DTYPE_F32)
                rows_store<float, N>(args, tokens, scales, sm.stored, t0, kb0, nkb, warp - 2, lane);
            else if (args.x_type == TQ_DTYPE_F16)
                rows_store<__half, N>(args, tokens, scales, sm.stored, t0, kb0, nkb, warp - 2, lane);
            else
                rows_store<__nv_bfloat16, N>(args, tokens, scales, sm.stored, t0, kb0, nkb, warp - 2, lane);
        }
    }
    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int i = 0; i < nkb; ++i) {
                const int s = i % SH::kStages;
                if (i >= SH::kStages && !wait(&sm.empty[s], (i / SH::kStages - 1) & 1)) break;
                unsigned char *a = ring + s * SH::kStageBytes;
                const int x = (kb0 + i) * cols_per_kb;
                mbar_arrive_expect_tx(&sm.full[s], SH::kStageBytes);
                if (KIND == kSwiglu) {
                    tma_load_2d(a, &map_w0, x, tile * 64, &sm.full[s]);
                    tma_load_2d(a + 8192, &map_w1, x, tile * 64, &sm.full[s]);
                } else {
                    tma_load_2d(a, &map_w0, x, tile * kRowsM, &sm.full[s]);
                }
                if (KIND != kFp8Store) tma_load_2d(a + kRowsM * 128, &map_x, x, t0, &sm.full[s]);
                ++issued;
            }
            // every issued copy has landed before the ring is used for anything else
            for (int i = max(0, issued - SH::kStages); i < issued; ++i)
                mbar_wait_sleep(&sm.full[i % SH::kStages], (i / SH::kStages) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc(kRowsM, N, SH::kIsFp8 ? 0 : (args.out_type == TQ_DTYPE_BF16 ? 1 : 0), 0, 0);
            for (int i = 0; i < nkb; ++i) {
                const int s = i % SH::kStages, st = i % SH::kAccStages;
                if (!wait(&sm.full[s], (i / SH::kStages) & 1)) break;
                if (KIND == kFp8Store && !wait(&sm.stored[i], 0)) break;
                if (SH::kIsFp8 && i >= SH::kAccStages && !wait(&sm.acc_empty[st], (i / SH::kAccStages - 1) & 1)) break;
                tc_fence_after();
                const uint32_t base = smem_u32(ring + s * SH::kStageBytes);
                const uint64_t ad = umma_desc_sw128(base), bd = umma_desc_sw128(
                    KIND == kFp8Store ? smem_u32(tokens + i * (N * 128)) : base + kRowsM * 128);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (SH::kIsFp8) umma_e4m3(tmem + st * N, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                    else umma_f16(tmem, ad + 2 * k, bd + 2 * k, idesc, (i | k) != 0);
                }
                umma_commit(&sm.empty[s]);
                if (SH::kIsFp8) umma_commit(&sm.acc_full[st]);
            }
            if (KIND == kSwiglu) umma_commit(&sm.acc_full[0]);
        }
    } else if (warp >= 4) {
        const int q = warp & 3;
        const int row = 32 * q + lane;
        const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16);
        float *partial = reinterpret_cast<float *>(ring);
        if constexpr (KIND == kSwiglu) {
            if (wait(&sm.acc_full[0], 0)) {
                tc_fence_after();
#pragma unroll
                for (int c0 = 0; c0 < N; c0 += 16) {
                    uint32_t v[16];
                    tmem_ld16(taddr + c0, v);
#pragma unroll
                    for (int c = 0; c < 16; ++c) partial[(c0 + c) * kRowsM + row] = __uint_as_float(v[c]);
                }
            }
        } else {
            float acc[N];
#pragma unroll
            for (int c = 0; c < N; ++c) acc[c] = 0.f;
            const int et = threadIdx.x - 128;                     // 0..127: the token whose scale it loads
            const bool mine = et < N && t0 + et < args.rows;
            const float *sx = args.sx + (size_t)(mine ? t0 + et : 0) * args.kblocks + kb0;
            const float *sw = args.sw + (size_t)tile * args.kblocks + kb0;
            float next = 0.f;
            if (nkb > 0) next = KIND == kFp8Store ? sw[0] : (mine ? sx[0] : 0.f) * sw[0];
            for (int i = 0; i < nkb; ++i) {
                const int st = i % SH::kAccStages;
                const float w = next;
                const float *slot = scales + (KIND == kFp8Store ? i : st) * N;
                if constexpr (KIND == kFp8Store) {
                    if (i + 1 < nkb) next = sw[i + 1];
                } else {
                    // the scales of this block; the slot's last readers are past the barrier
                    // of block i - 1
                    if (et < N) scales[st * N + et] = w;
                    if (i + 1 < nkb) next = (mine ? sx[i + 1] : 0.f) * sw[i + 1];
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                }
                // The token scales come from the storing warps' own stores, which the MMA's commit
                // does not order: their barrier does (looked at under the MMAs of the block).
                bool got = true;
                if (KIND == kFp8Store) got = wait(&sm.stored[i], 0);
                got = got && wait(&sm.acc_full[st], (i / SH::kAccStages) & 1);
                const bool ok = __all_sync(0xffffffffu, got);
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < N; c0 += 16) {
                        uint32_t v[16];
                        tmem_ld16(taddr + st * N + c0, v);
                        const float4 *sc = reinterpret_cast<const float4 *>(slot + c0);
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            float4 f = sc[c >> 2];
                            if (KIND == kFp8Store) {
                                f.x *= w; f.y *= w; f.z *= w; f.w *= w;
                            }
                            acc[c0 + c] = fmaf(f.x, __uint_as_float(v[c]), acc[c0 + c]);
                            acc[c0 + c + 1] = fmaf(f.y, __uint_as_float(v[c + 1]), acc[c0 + c + 1]);
                            acc[c0 + c + 2] = fmaf(f.z, __uint_as_float(v[c + 2]), acc[c0 + c + 2]);
                            acc[c0 + c + 3] = fmaf(f.w, __uint_as_float(v[c + 3]), acc[c0 + c + 3]);
                        }
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.acc_empty[st]);
            }
            // the last acc_full completed: every MMA has read the ring
#pragma unroll
            for (int c = 0; c < N; ++c) partial[c * kRowsM + row] = acc[c];
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();                       // every CTA's partial sums are in its ring
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, SH::kTmemCols);
    }

    // rank r adds the tokens [r N / C, (r + 1) N / C) over the CTAs, in rank order
    const int per = N / C;
    const uint32_t ring_s = smem_u32(ring);
    constexpr int kQuads = KIND == kSwiglu ? 16 : 32;    // groups of 4 outputs per token
    for (int i = threadIdx.x; i < per * kQuads; i += kRowsThreads) {
        const int c = rank * per + i / kQuads, o = (i % kQuads) * 4;
        const int t = t0 + c;
        if (t >= args.rows) continue;
        float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < C; ++p) {
            const uint32_t at = map_to_rank(ring_s + (uint32_t)(c * kRowsM + o) * 4u, p);
            const float4 v = ld_cluster_f4(at);
            a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
            if (KIND == kSwiglu) {
                const float4 w = ld_cluster_f4(at + 64u * 4u);
                b[0] += w.x; b[1] += w.y; b[2] += w.z; b[3] += w.w;
            }
        }
        const int col = tile * (KIND == kSwiglu ? 64 : kRowsM) + o;
        if (col >= args.width) continue;
        if (KIND == kSwiglu) {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = swiglu_value(a[j], b[j]);
        }
        store_out4(args.out, (size_t)t * args.width + col, a, min(4, args.width - col), args.out_type,
                   args.accumulate != 0);
    }
    cluster_sync_all();                       // no CTA leaves while another reads its ring
}

// Cluster size of the K split: the most CTAs a tile that leave every SM one CTA, or two
// where only two are to be had by it (and both fit).  More CTAs than that cost more in
// partial sums than they bring: 203 tokens, 2056 -> 1000, C = 4 (128 CTAs) 8.7 us, C = 8
// 12.6; 16 tokens, 4096 -> 16384 in E4M3, C = 1, 2, 4: 14.3, 10.9, 14.5.  A SwiGLU tile of 128
// tokens has 64 KB of partial sums a CTA: 4 CTAs 9.5 us, 8 CTAs 11.1 (128 tokens, 4096 -> 1024).
template <int N, int KIND>
inline int rows_cluster(long long tiles, int kblocks) {
    const bool two = KIND == kSwiglu || N <= 64;
    int c = KIND == kSwiglu && N > 64 ? 4 : 8;
    while (c > 1 && (tiles * c > (c == 2 && two ? 2LL : 1LL) * num_sms() || c > kblocks)) c >>= 1;
    return c;
}

// K-blocks of a CTA with one token tile of N rows.
template <int N>
inline int rows_share(int width, int kblocks) {
    const int c = rows_cluster<N, kFp8Store>((width + (long long)kRowsM - 1) / kRowsM, kblocks);
    return (kblocks + c - 1) / c;
}

template <int N, int KIND>
static bool configure_rows() {
    return set_smem(dense_rows_kernel<N, KIND>, RowsShape<N, KIND>::kBytes);
}

template <int N, int KIND>
static int launch_rows(const CUtensorMap &w0, const CUtensorMap &w1, const CUtensorMap &x, const RowsArgs &a,
                       cudaStream_t s, bool chained) {
    using SH = RowsShape<N, KIND>;
    const int per_tile = KIND == kSwiglu ? 64 : kRowsM;
    const long long row_tiles = (a.width + (long long)per_tile - 1) / per_tile;
    const int token_tiles = (a.rows + N - 1) / N;
    const int c = rows_cluster<N, KIND>(row_tiles * token_tiles, a.kblocks);
    cudaError_t e = launch_cluster(dense_rows_kernel<N, KIND>, dim3((unsigned)(row_tiles * c), token_tiles),
                                   dim3(kRowsThreads), SH::kBytes, s, c, chained, w0, w1, x, a);
    return e == cudaSuccess ? launch_status() : record_cuda_error("dense_rows_kernel");
}

}  // namespace tq
