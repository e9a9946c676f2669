// E4M3 with a scale for each block of 128: storage (rows in 1 x 128 blocks, weights in
// 128 x 128 blocks) and the matrix product
//
//   y[m][n] = sum_b s_x[m][b] s_w[n / 128][b] sum_{k in block b} x8[m][k] w8[n][k]
//
// A block's scale is the power of two 2^e, e = min { e >= -126 : max|x| <= 448 * 2^e }
// over its finite values, so scaling is exact and storing costs one rounding, to E4M3.
// The product takes any fp32 scales.
//
// The product of many rows (fp8_pair_kernel): a CTA pair owns a 256 x 256 tile.  A K-block
// of 128 bytes is one scale block: its 4 MMAs (256 x 256 x 32, kind::f8f6f4) write a fresh
// fp32 accumulator in tensor memory, and while the next block's MMAs fill the other one
// the 8 epilogue warps of each CTA add s_x s_w times it to fp32 registers (128 columns of
// a row a thread).  Per CTA and K-block the MMAs take 512 cycles at the E4M3 rate, reading
// 128 x 256 accumulators and as many FMAs at least 256 each on their own pipes.  Measured
// (8192 x 4096 x 4096, 130 us): 1050 a K-block, 840 without the FMAs, the tensor pipe busy 47 %; both
// accumulators fill tensor memory, so the MMAs of block k + 2 wait until all 16 warps have read block k.
// Few rows: dense_rows_kernel.
#include "tq_dense_rows.cuh"

namespace tq {

// ------------------------------------------------------------------------------ storage

// Row kernels: a warp takes kStoreRows rows of 512 columns (4 blocks), 16 lanes a block,
// 8 values a lane; blockIdx.y is the group of 512 columns, so no index is divided.  All
// loads of a warp are in flight together (4 a lane), which the reads from HBM need.
constexpr int kStoreRows = 2;
constexpr int kStoreWarps = 8;

// 1 x 128 blocks: a row's values are read once and its largest magnitude takes 4 exchanges.
// Memory-bound.
template <typename T>
__global__ void __launch_bounds__(kStoreWarps * 32) fp8_quantize_rows_kernel(const T *x, long long rows,
                                                                            int cols, uint8_t *out,
                                                                            float *scales) {
    chain_entry();
    const int nb = (cols + 127) / 128;
    const int lane = threadIdx.x & 31;
    const long long r0 = ((long long)blockIdx.x * kStoreWarps + (threadIdx.x >> 5)) * kStoreRows;
    const int c0 = blockIdx.y * 512 + lane * 8;
    float v[kStoreRows][2][8];
#pragma unroll
    for (int k = 0; k < kStoreRows; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 256 * h;
            if (r0 + k < rows && c < cols) load8<T>(x + (size_t)(r0 + k) * cols + c, v[k][h]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) v[k][h][j] = 0.f;
        }
#pragma unroll
    for (int k = 0; k < kStoreRows; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 256 * h;
            float s;
            const uint2 q = fp8_store_block(v[k][h], s);
            if (r0 + k < rows && c < cols) {
                *reinterpret_cast<uint2 *>(out + (size_t)(r0 + k) * cols + c) = q;
                if ((lane & 15) == 0) scales[(size_t)(r0 + k) * nb + c / 128] = s;
            }
        }
}

// 128 x 128 blocks: one CTA a block, 64 values a thread kept in registers.
template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_blocks_kernel(const T *x, long long rows, int cols,
                                                                  uint8_t *out,
                                                                  float *scales) {
    chain_entry();
    __shared__ float warp_max[8];
    const int nb = (cols + 127) / 128;
    const long long rb = blockIdx.x / nb;
    const int b = (int)(blockIdx.x - rb * nb);
    const int c = b * 128 + (threadIdx.x & 15) * 8;
    float v[8][8];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long r = rb * 128 + i * 16 + (threadIdx.x >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        if (r < rows && c < cols) load8<T>(x + (size_t)r * cols + c, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = finite_max(m, v[i][j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, warp_max[i]);
    const int e = e4m3_block_exponent(m);
    const float inv = exp2_int(-e);
    if (threadIdx.x == 0) scales[blockIdx.x] = exp2_int(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long r = rb * 128 + i * 16 + (threadIdx.x >> 4);
        if (r < rows && c < cols)
            *reinterpret_cast<uint2 *>(out + (size_t)r * cols + c) =
                make_uint2(e4m3x4_scaled(v[i][0], v[i][1], v[i][2], v[i][3], inv),
                           e4m3x4_scaled(v[i][4], v[i][5], v[i][6], v[i][7], inv));
    }
}

// Stored values times their scales, laid out over warps as the row kernel above: block
// (bx, by) of store_grid.  Memory-bound.
__device__ __forceinline__ void fp8_dequantize_block(long long bx, int by, const uint8_t *q,
                                                     const float *scales, long long rows, int cols,
                                                     int block_rows, void *out, int type) {
    const int nb = (cols + 127) / 128;
    const long long r0 = (bx * kStoreWarps + (threadIdx.x >> 5)) * kStoreRows;
    const int c0 = by * 512 + (threadIdx.x & 31) * 8;
    uint2 w[kStoreRows][2];
    float s[kStoreRows][2];
#pragma unroll
    for (int k = 0; k < kStoreRows; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 256 * h;
            if (r0 + k < rows && c < cols) {
                w[k][h] = *reinterpret_cast<const uint2 *>(q + (size_t)(r0 + k) * cols + c);
                s[k][h] = scales[(size_t)(block_rows == 1 ? r0 + k : (r0 + k) / 128) * nb + c / 128];
            }
        }
#pragma unroll
    for (int k = 0; k < kStoreRows; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = c0 + 256 * h;
            if (r0 + k >= rows || c >= cols) continue;
            float v[8];
            e4m3x4_to_f32(w[k][h].x, *reinterpret_cast<float(*)[4]>(v));
            e4m3x4_to_f32(w[k][h].y, *reinterpret_cast<float(*)[4]>(v + 4));
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= s[k][h];
            const size_t at = (size_t)(r0 + k) * cols + c;
            if (type == TQ_DTYPE_F32) {
                float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + at);
                p[0] = make_float4(v[0], v[1], v[2], v[3]);
                p[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                const bool f16 = type == TQ_DTYPE_F16;
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + at) =
                    make_uint4(pack16(v[0], v[1], f16), pack16(v[2], v[3], f16), pack16(v[4], v[5], f16),
                               pack16(v[6], v[7], f16));
            }
        }
}

__global__ void __launch_bounds__(kStoreWarps * 32) fp8_dequantize_kernel(const uint8_t *q,
                                                                         const float *scales,
                                                                         long long rows, int cols, int block_rows,
                                                                         void *out, int type) {
    chain_entry();
    fp8_dequantize_block(blockIdx.x, blockIdx.y, q, scales, rows, cols, block_rows, out, type);
}

// ------------------------------------------------------------------------------ product

constexpr int kFp8Stages = 5;
constexpr int kFp8Threads = 384;       // warp 0 TMA, 1 MMA (leader), 2 TMEM, 4-11 epilogue
constexpr int kFp8StageBytes = 16384;  // 128 rows x 128 E4M3

struct __align__(1024) Fp8Smem {
    unsigned char a[kFp8Stages][kFp8StageBytes];
    unsigned char b[kFp8Stages][kFp8StageBytes];
    unsigned char rows[8][kRowStage];
    float scales[8][256];           // [K-block mod 8][accumulating thread]: its row's s_x s_w
    uint64_t full[kFp8Stages];      // leader: both CTAs' copies of the stage
    uint64_t empty[kFp8Stages];     // MMA commit, in both CTAs
    uint64_t acc_full[2];           // MMA commit, in both CTAs
    uint64_t acc_empty[2];          // leader: the 16 epilogue warps of the pair
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(Fp8Smem) + 1024 <= 227 * 1024, "E4M3 pair GEMM shared memory");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFp8Threads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                    const RowsArgs args) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    Fp8Smem &sm = *reinterpret_cast<Fp8Smem *>(smem_raw + pad);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int m_tiles = (args.rows + 255) / 256, n_tiles = (args.width + 255) / 256;
    const long long tiles = (long long)m_tiles * n_tiles;
    const long long pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int nkb = args.kblocks;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kFp8Stages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], 16);
        }
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc_pair(&sm.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
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

    // Registers: 384 threads are launched with 168 each (64,512); 4 warps of 56 and 8 of 224
    // are 64,512.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0 && lane == 0) {
            bool ok = true;
            uint32_t it = 0;
            for (long long t = pair; t < tiles && ok; t += pairs) {
                int m, n;
                grouped_tile(t, m_tiles, n_tiles, m, n);
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int s = it % kFp8Stages;
                    if (it >= kFp8Stages && !wait(&sm.empty[s], (it / kFp8Stages - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = map_to_rank(smem_u32(&sm.full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 4 * kFp8StageBytes);
                    tma_load_2d_pair(sm.a[s], &map_a, kb * 128, m * 256 + 128 * rank, bar);
                    tma_load_2d_pair(sm.b[s], &map_b, kb * 128, n * 256 + 128 * rank, bar);
                }
            }
            for (uint32_t i = it > kFp8Stages ? it - kFp8Stages : 0; i < it && ok; ++i)
                ok = wait(&sm.empty[i % kFp8Stages], (i / kFp8Stages) & 1);
            if (!ok)       // a wait gave up: time for the copies in flight to land
                for (int i = 0; i < 2000; ++i) __nanosleep(1000);
        } else if (warp == 1 && rank == 0 && lane == 0) {
            const uint32_t idesc = umma_idesc(256, 256, 0, 0, 0);
            bool ok = true;
            uint32_t it = 0;
            for (long long t = pair; t < tiles && ok; t += pairs) {
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const int s = it % kFp8Stages;
                    const uint32_t st = it & 1, d = tmem + st * 256;
                    if (!wait(&sm.full[s], (it / kFp8Stages) & 1) ||
                        (it >= 2 && !wait(&sm.acc_empty[st], ((it >> 1) - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = umma_desc_sw128(smem_u32(sm.a[s])), bd = umma_desc_sw128(smem_u32(sm.b[s]));
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_e4m3_pair(d, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                    umma_commit_pair(&sm.empty[s]);
                    umma_commit_pair(&sm.acc_full[st]);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int q = warp & 3, w = (warp - 4) >> 2;
        const int row = 128 * rank + 32 * q + lane;
        const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + 128 * w;
        const int n_blocks = (args.width + 127) / 128;
        uint32_t it = 0;
        bool ok = true;
        for (long long t = pair; t < tiles && ok; t += pairs) {
            int m, n;
            grouped_tile(t, m_tiles, n_tiles, m, n);
            const int r = m * 256 + row, nb = n * 2 + w;
            const bool mine = r < args.rows && nb < n_blocks;
            const float *sx = args.sx + (size_t)(mine ? r : 0) * nkb;
            const float *sw = args.sw + (size_t)(mine ? nb : 0) * nkb;
            uint64_t acc[64];          // pairs of columns
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            // The blocks' scales: four at a time, loaded four blocks ahead, multiplied and kept
            // in a place of the thread's own (a load for each block cost 4 of 139 us at
            // 8192 x 4096 x 4096).
            float *place = &sm.scales[0][threadIdx.x - 128];
            float4 gx, gw;
            auto load_group = [&](int k) {
                gx = gw = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!mine || k >= nkb) return;
                if ((nkb & 3) == 0) {
                    gx = *reinterpret_cast<const float4 *>(sx + k);
                    gw = *reinterpret_cast<const float4 *>(sw + k);
                } else {
                    gx.x = sx[k]; gw.x = sw[k];
                    if (k + 1 < nkb) { gx.y = sx[k + 1]; gw.y = sw[k + 1]; }
                    if (k + 2 < nkb) { gx.z = sx[k + 2]; gw.z = sw[k + 2]; }
                    if (k + 3 < nkb) { gx.w = sx[k + 3]; gw.w = sw[k + 3]; }
                }
            };
            load_group(0);
            for (int kb = 0; kb < nkb; ++kb, ++it) {
                const uint32_t st = it & 1;
                if ((kb & 3) == 0) {
                    float *p = place + (kb & 4) * 256;
                    p[0] = gx.x * gw.x;
                    p[256] = gx.y * gw.y;
                    p[512] = gx.z * gw.z;
                    p[768] = gx.w * gw.w;
                    load_group(kb + 4);
                }
                const float f1 = place[(kb & 7) * 256];
                const uint64_t f = f32x2(f1, f1);
                ok = __all_sync(0xffffffffu, wait(&sm.acc_full[st], (it >> 1) & 1));
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = taddr + st * 256;
                uint32_t a[32], b[32];
                // two loads in flight a wait: a load's latency, not its bandwidth, is what a
                // warp waits for
                tmem_ld32(at, a);
                tmem_ld32(at + 32, b);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) fma_f32x2(acc[i], f, a[2 * i], a[2 * i + 1]);
#pragma unroll
                for (int i = 0; i < 16; ++i) fma_f32x2(acc[16 + i], f, b[2 * i], b[2 * i + 1]);
                tmem_ld32(at + 64, a);
                tmem_ld32(at + 96, b);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(map_to_rank(smem_u32(&sm.acc_empty[st]), 0));
#pragma unroll
                for (int i = 0; i < 16; ++i) fma_f32x2(acc[32 + i], f, a[2 * i], a[2 * i + 1]);
#pragma unroll
                for (int i = 0; i < 16; ++i) fma_f32x2(acc[48 + i], f, b[2 * i], b[2 * i + 1]);
            }
            if (!ok) break;
            // the warp's 32 rows x 128 columns, 128 bytes of each row at a time
            const int col = n * 256 + 128 * w, row0 = m * 256 + 128 * rank + 32 * q;
            const int es = args.out_type == TQ_DTYPE_F32 ? 4 : 2;
            const size_t row_bytes = (size_t)args.width * es;
            const bool vec16 = row_bytes % 16 == 0;
            char *out = reinterpret_cast<char *>(args.out) + (size_t)row0 * row_bytes + (size_t)col * es;
            const int bytes = (args.width - col < 128 ? args.width - col : 128) * es, rows = args.rows - row0;
            uint4 v[8];
            if (es == 4) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint64_t x = acc[16 * c + 2 * i], y = acc[16 * c + 2 * i + 1];
                        v[i] = make_uint4((uint32_t)x, (uint32_t)(x >> 32), (uint32_t)y, (uint32_t)(y >> 32));
                    }
                    warp_store_rows<4>(sm.rows[warp - 4], lane, v, out + 128 * c, row_bytes, rows, bytes - 128 * c,
                                       vec16, args.accumulate != 0);
                }
            } else {
                const bool f16 = args.out_type == TQ_DTYPE_F16;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t p[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t x = acc[32 * c + 4 * i + j];
                            p[j] = pack16(f32x2_lo(x), f32x2_hi(x), f16);
                        }
                        v[i] = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    warp_store_rows<2>(sm.rows[warp - 4], lane, v, out + 128 * c, row_bytes, rows, bytes - 128 * c,
                                       vec16);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ------------------------------------------------------------------------------ host side

// Rows the weight-streaming kernel takes: up to 128 (it is bound by reading w), and as many
// more as leave a cluster of two CTAs a tile of 128 rows by 128 outputs, one CTA a SM: a pair
// of the other kernel then has too few tiles (333 x 1001 x 2064: 8.4 us here, 13.2 there; 333 x
// 4096 x 4096, 96 tiles: 21.9 here, 20.9 there).
static bool fp8_rows_case(int M, int N) {
    if (M <= 128) return true;
    return 2 * ((M + 127LL) / 128) * ((N + 127LL) / 128) <= num_sms();
}

// Whether the product stores its activations itself (one launch, no workspace): every CTA
// then stores its share of K for all tokens, which pays up to 128 blocks of a row (1 x 4096 x
// 4096: 8 blocks, 6.4 us against 7.4 in two launches; 16 x 4096 x 4096: 128 blocks, 8.3 against
// 8.4; 16 x 16384 x 4096: 256 blocks, 21.6 against 16.6).
static bool fp8_fused_case(int M, int N, int K) {
    if (M > 16) return false;
    const int share = rows_share<16>(N, (K + 127) / 128);
    return share <= RowsStore<16>::kMost && M * share <= 128;
}

static bool configure_store() {
    return set_smem(fp8_quantize_rows_kernel<__half>, 0) || set_smem(fp8_quantize_rows_kernel<__nv_bfloat16>, 0) ||
           set_smem(fp8_quantize_rows_kernel<float>, 0);
}

// The first product on a device sets up every kernel that a later one may launch (their launch
// attributes; loading them), so that later calls may be captured.
static int configure_fp8() {
    static PerDeviceFlag configured;
    if (configured.get()) return TQ_OK;
    if (set_smem(fp8_pair_kernel, (int)sizeof(Fp8Smem) + 1024) || configure_rows<16, kFp8>() ||
        configure_rows<32, kFp8>() || configure_rows<64, kFp8>() || configure_rows<128, kFp8>() ||
        configure_rows<16, kFp8Store>() || configure_store())
        return record_cuda_error("configure_fp8");
    configured.set();
    return TQ_OK;
}

static int fp8_product(const uint8_t *x8, const float *sx, const uint8_t *w8, const float *sw, int M, int N, int K,
                       void *y, int y_dtype, int accumulate, cudaStream_t s) {
    RowsArgs a{};
    a.rows = M;
    a.width = N;
    a.kblocks = (K + 127) / 128;
    a.out_type = y_dtype;
    a.accumulate = accumulate;
    a.out = y;
    a.sx = sx;
    a.sw = sw;
    CUtensorMap mw, mx;
    const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    int st = matrix_map(&mw, u8, 1, w8, N, K, 128);
    if (st) return st;
    if (fp8_rows_case(M, N)) {
        const int n = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
        st = matrix_map(&mx, u8, 1, x8, M, K, n);
        if (st) return st;
        LaunchScope ls(s, kStageFp8Gemm);
        switch (n) {
            case 16: return launch_rows<16, kFp8>(mw, mw, mx, a, s, true);
            case 32: return launch_rows<32, kFp8>(mw, mw, mx, a, s, true);
            case 64: return launch_rows<64, kFp8>(mw, mw, mx, a, s, true);
            default: return launch_rows<128, kFp8>(mw, mw, mx, a, s, true);
        }
    }
    st = matrix_map(&mx, u8, 1, x8, M, K, 128);
    if (st) return st;
    const int smem = (int)sizeof(Fp8Smem) + 1024;
    const long long tiles = ((M + 255LL) / 256) * ((N + 255LL) / 256), pairs = num_sms() / 2;
    LaunchScope ls(s, kStageFp8Gemm);
    if (launch_chained(fp8_pair_kernel, dim3(2 * (unsigned)(tiles < pairs ? tiles : pairs)), dim3(kFp8Threads), smem, s,
                       mx, mw, a) != cudaSuccess)
        return record_cuda_error("fp8_pair_kernel");
    return launch_status();
}

// The product of few rows from activations of 16 or 32 bits, one launch.
static int fp8_product_fused(const void *x, int x_dtype, const uint8_t *w8, const float *sw, int M, int N, int K,
                             void *y, int y_dtype, int accumulate, cudaStream_t s) {
    RowsArgs a{};
    a.rows = M;
    a.width = N;
    a.kblocks = (K + 127) / 128;
    a.out_type = y_dtype;
    a.accumulate = accumulate;
    a.out = y;
    a.sw = sw;
    a.x = x;
    a.cols = K;
    a.x_type = x_dtype;
    CUtensorMap mw;
    const int st = matrix_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w8, N, K, 128);
    if (st) return st;
    LaunchScope ls(s, kStageFp8Gemm);
    return launch_rows<16, kFp8Store>(mw, mw, mw, a, s, true);
}

// Shape and type checks of a product; 0 rows or outputs is a valid no-op.
static int fp8_product_status(int M, int N, int K, int y_dtype, int accumulate) {
    if (M < 0 || N < 0 || K < 1 || K % 16) return TQ_ERR_INVALID_ARG;
    if (y_dtype < TQ_DTYPE_F16 || y_dtype > TQ_DTYPE_F32) return TQ_ERR_INVALID_ARG;
    if (accumulate && y_dtype != TQ_DTYPE_F32) return TQ_ERR_UNSUPPORTED;
    if (M > kMostSize || N > kMostSize || K > kMostSize) return TQ_ERR_UNSUPPORTED;
    return TQ_OK;
}

// Grid of the row kernels, and whether it is one.
static dim3 store_grid(long long rows, int cols) {
    const long long per = kStoreWarps * kStoreRows;
    return dim3((unsigned)((rows + per - 1) / per), (unsigned)((cols + 511) / 512));
}
static bool store_grid_fits(long long rows, int cols) {
    return rows <= 0x7FFFFFFFLL * kStoreWarps * kStoreRows && ((long long)cols + 511) / 512 <= 65535;
}

template <typename T>
static cudaError_t quantize_launch(const void *x, long long rows, int cols, int block_rows, uint8_t *out, float *scales,
                                   cudaStream_t s) {
    const long long nb = (cols + 127LL) / 128;
    if (block_rows == 1)
        return launch_chained(fp8_quantize_rows_kernel<T>, store_grid(rows, cols),
                              dim3(kStoreWarps * 32), 0, s,
                              (const T *)x, rows, cols, out, scales);
    return launch_chained(fp8_quantize_blocks_kernel<T>, dim3((unsigned)((rows + 127) / 128 * nb)), dim3(256), 0, s,
                          (const T *)x, rows, cols, out, scales);
}

}  // namespace tq

TQ_API int fp8_block_quantize(const void *x, int x_dtype, int64_t rows, int cols, int block_rows, uint8_t *out,
                              float *scales, tq_stream stream) {
    using namespace tq;
    if (x_dtype < TQ_DTYPE_F16 || x_dtype > TQ_DTYPE_F32 || rows < 0 || cols < 1 || cols % 8 ||
        (block_rows != 1 && block_rows != 128))
        return TQ_ERR_INVALID_ARG;
    if (cols > kMostSize) return TQ_ERR_UNSUPPORTED;
    if (rows == 0) return TQ_OK;
    if (block_rows == 128 ? (rows + 127) / 128 * ((cols + 127LL) / 128) > 0x7FFFFFFFLL : !store_grid_fits(rows, cols))
        return TQ_ERR_UNSUPPORTED;
    if (!x || !out || !scales) return TQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(out) || !aligned16(scales)) return TQ_ERR_ALIGNMENT;
    const cudaStream_t s = (cudaStream_t)stream;
    LaunchScope ls(s, kStageFp8Store);
    const cudaError_t e = x_dtype == TQ_DTYPE_F16    ? quantize_launch<__half>(x, rows, cols, block_rows, out, scales, s)
                          : x_dtype == TQ_DTYPE_BF16 ? quantize_launch<__nv_bfloat16>(x, rows, cols, block_rows, out, scales, s)
                                                     : quantize_launch<float>(x, rows, cols, block_rows, out, scales, s);
    return e == cudaSuccess ? launch_status() : record_cuda_error("fp8_block_quantize");
}

TQ_API int fp8_block_dequantize(const uint8_t *q, const float *scales, int64_t rows, int cols, int block_rows, void *out,
                                int out_dtype, tq_stream stream) {
    using namespace tq;
    if (out_dtype < TQ_DTYPE_F16 || out_dtype > TQ_DTYPE_F32 || rows < 0 || cols < 1 || cols % 8 ||
        (block_rows != 1 && block_rows != 128))
        return TQ_ERR_INVALID_ARG;
    if (cols > kMostSize) return TQ_ERR_UNSUPPORTED;
    if (rows == 0) return TQ_OK;
    if (!store_grid_fits(rows, cols)) return TQ_ERR_UNSUPPORTED;
    if (!q || !scales || !out) return TQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(scales) || !aligned16(out)) return TQ_ERR_ALIGNMENT;
    const cudaStream_t s = (cudaStream_t)stream;
    LaunchScope ls(s, kStageFp8Store);
    if (launch_chained(fp8_dequantize_kernel, store_grid(rows, cols), dim3(kStoreWarps * 32), 0, s, q, scales,
                       (long long)rows, cols, block_rows, out, out_dtype) != cudaSuccess)
        return record_cuda_error("fp8_block_dequantize");
    return launch_status();
}

TQ_API int fp8_block_gemm(const uint8_t *x, const float *s_x, const uint8_t *w, const float *s_w, int M, int N, int K,
                          void *y, int y_dtype, int accumulate, tq_stream stream) {
    using namespace tq;
    const int st = fp8_product_status(M, N, K, y_dtype, accumulate);
    if (st || M == 0 || N == 0) return st;
    if (!x || !s_x || !w || !s_w || !y) return TQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(s_x) || !aligned16(s_w)) return TQ_ERR_ALIGNMENT;
    if (const int c = configure_fp8()) return c;
    return fp8_product(x, s_x, w, s_w, M, N, K, y, y_dtype, accumulate, (cudaStream_t)stream);
}

TQ_API size_t fp8_block_linear_workspace_size(int M, int N, int K) {
    if (tq::fp8_product_status(M, N, K, TQ_DTYPE_F32, 0) || M == 0 || N == 0 || tq::fp8_fused_case(M, N, K)) return 0;
    const size_t q = ((size_t)M * K + 255) & ~(size_t)255;
    return q + (((size_t)M * ((K + 127) / 128) * 4 + 255) & ~(size_t)255);
}

TQ_API int fp8_block_linear(const void *x, int x_dtype, const uint8_t *w, const float *s_w, int M, int N, int K, void *y,
                            int y_dtype, int accumulate, void *ws, size_t ws_bytes, tq_stream stream) {
    using namespace tq;
    int st = fp8_product_status(M, N, K, y_dtype, accumulate);
    if (!st && (x_dtype < TQ_DTYPE_F16 || x_dtype > TQ_DTYPE_F32)) st = TQ_ERR_INVALID_ARG;
    if (st || M == 0 || N == 0) return st;
    if (!x || !w || !s_w || !y) return TQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(s_w) || (ws && !aligned16(ws)))
        return TQ_ERR_ALIGNMENT;
    const bool fused = fp8_fused_case(M, N, K);
    if (!fused && (!ws || ws_bytes < fp8_block_linear_workspace_size(M, N, K))) return TQ_ERR_WORKSPACE;
    if ((st = configure_fp8())) return st;
    if (fused)
        return fp8_product_fused(x, x_dtype, w, s_w, M, N, K, y, y_dtype, accumulate, (cudaStream_t)stream);
    uint8_t *q = reinterpret_cast<uint8_t *>(ws);
    float *sx = reinterpret_cast<float *>(q + (((size_t)M * K + 255) & ~(size_t)255));
    st = fp8_block_quantize(x, x_dtype, M, K, 1, q, sx, stream);
    if (st) return st;
    return fp8_product(q, sx, w, s_w, M, N, K, y, y_dtype, accumulate, (cudaStream_t)stream);
}
