// Shared pieces of the dense (not trellis-coded) operators: CTA-pair tcgen05 helpers,
// cluster helpers, tensor maps of row-major matrices, E4M3 block scaling.
//
// The kernels are launched chained (a kernel may start before the one before it has ended, and
// waits in chain_entry), so what they read may still be written while they start: no pointer is
// declared __restrict__ and no load goes through the read-only path.
#pragma once

#include "tq_common.cuh"

#include <cuda.h>
#include <float.h>

namespace tq {

// Stage tags of this file's users (tq_profile_*), after those of Stage.
constexpr int kStageSwiglu = kNumStages, kStageSwigluGrad = kNumStages + 1, kStageFp8Store = kNumStages + 2,
              kStageFp8Gemm = kNumStages + 3;
static_assert(kStageSwiglu == 15, "the C header documents the numbers");

// ------------------------------------------------------------------------------ cluster

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Every thread of every CTA of the cluster; orders shared-memory accesses before it (in
// any CTA) against those after it.
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address, in the cluster's shared-memory window, of CTA `rank`'s copy of `saddr`.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Arrival on a barrier of another CTA that hands over tensor memory which this thread has
// finished reading (its loads waited for): no generic memory is handed over, so it needs no
// release, whose cluster-wide fence stalled the accumulator loop (8192 x 4096 x 4096 in E4M3:
// 311 us with it, 195 without).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// One look at a barrier, without the wait that a try_wait may take.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// ------------------------------------------------------------------------------ CTA pair

// Tensor copy into this CTA's shared memory whose bytes complete on a barrier of either
// CTA of the pair (`bar` is an address of the cluster's window).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` (same offset) of both CTAs once the issued MMAs have completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst_smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

// 32 lanes x 32 consecutive 32-bit columns, without the wait (tmem_ld_wait).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// MN-major operand in shared memory with the 128-byte swizzle, as a tensor copy with a
// box of 64 (MN) x 64 (K) 16-bit elements lays it out: K rows of 128 bytes, 8-row atoms
// 1024 B apart (SBO), the next 64 MN elements one 8 KB box further (LBO).  A K = 16 step
// is two atoms, 2048 B.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(8192u >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// Instruction descriptor: fp32 D, operand format `fmt` for both operands (kind::f16: 0
// fp16, 1 bf16; kind::f8f6f4: 0 E4M3), a_mn / b_mn 1 for an MN-major operand.
__host__ __device__ constexpr uint32_t umma_idesc(int m, int n, int fmt, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)fmt << 7) | ((uint32_t)fmt << 10) | ((uint32_t)a_mn << 15) |
           ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ------------------------------------------------------------------------------ E4M3 blocks

// Exponent of a block's scale 2^e, e = min { e >= -126 : m <= 448 * 2^e }, from its
// largest finite magnitude m (0 for an all-zero block).  448 = 1.75 * 2^8.
__device__ __forceinline__ int e4m3_block_exponent(float m) {
    if (!(m > 0.f)) return 0;
    const uint32_t b = __float_as_uint(m);
    return max(-126, (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0));
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 <= e <= 127

// Largest magnitude over finite values: an infinity or NaN does not set a block's scale.
__device__ __forceinline__ float finite_max(float m, float v) {
    const float a = fabsf(v);
    return a <= FLT_MAX ? fmaxf(m, a) : m;
}

// Two values as E4M3 bytes (nearest even); the low byte is v0.  fma(y, 0, y) leaves a
// finite y as it is and makes an infinity NaN, which E4M3 can hold (it has no infinity,
// and the conversion alone would store 448).
__device__ __forceinline__ uint32_t e4m3x2_scaled(float v0, float v1, float inv) {
    float a = v0 * inv, b = v1 * inv;
    a = fmaf(a, 0.f, a);
    b = fmaf(b, 0.f, b);
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
    return d;
}

__device__ __forceinline__ uint32_t e4m3x4_scaled(float v0, float v1, float v2, float v3, float inv) {
    return e4m3x2_scaled(v0, v1, inv) | (e4m3x2_scaled(v2, v3, inv) << 16);
}

// Four E4M3 bytes as fp32 (exact: every E4M3 value is an fp16 value).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t q, float (&v)[4]) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(q & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(q >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

// ------------------------------------------------------------------------------ fp32 pairs

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float f32x2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f32x2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// acc += f * (lo, hi): two fp32 FMAs (nearest even) in one instruction.
__device__ __forceinline__ void fma_f32x2(uint64_t &acc, uint64_t f, uint32_t lo, uint32_t hi) {
    asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%2, %3};\n\tfma.rn.f32x2 %0, %1, v, %0;\n\t}"
        : "+l"(acc)
        : "l"(f), "r"(lo), "r"(hi));
}

// ------------------------------------------------------------------------------ 16-bit packing

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack16(float a, float b, bool f16) { return f16 ? pack_f16(a, b) : pack_bf16(a, b); }

// ------------------------------------------------------------------------------ row stores

// An accumulator thread holds a row, so its own stores would touch 32 rows an instruction
// and write a 32-byte sector in two to four pieces.  A warp instead passes 32 rows x 128
// bytes through shared memory (16-byte chunk i of row r at chunk i ^ (r mod 8): no bank conflicts)
// and stores four whole 128-byte row pieces an instruction.
constexpr int kRowStage = 32 * 128;      // bytes a warp

// Place of byte c of row r in a warp's stage.
__device__ __forceinline__ int row_stage_at(int r, int c) { return r * 128 + ((((c >> 4) ^ r) & 7) << 4) + (c & 15); }

// v: the lane's row (row `lane` of 32, 128 bytes); out: the warp's first row at its first
// byte; row_bytes: distance of rows; rows, bytes: how many of the 32 rows and 128 bytes exist.
// vec16: row_bytes and out are multiples of 16 (bytes then is, too).  ELEM: bytes of an
// element, stored one by one otherwise.  accumulate (fp32): add to what is there.
template <int ELEM>
__device__ __forceinline__ void warp_store_rows(unsigned char *stage, int lane, const uint4 (&v)[8], char *out,
                                                size_t row_bytes, int rows, int bytes, bool vec16,
                                                bool accumulate = false) {
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(stage + row_stage_at(lane, 16 * i)) = v[i];
    __syncwarp();
    if (vec16) {
        const int c = (lane & 7) * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            if (r < rows && c < bytes) {
                uint4 w = *reinterpret_cast<const uint4 *>(stage + row_stage_at(r, c));
                uint4 *p = reinterpret_cast<uint4 *>(out + (size_t)r * row_bytes + c);
                if (ELEM == 4 && accumulate) {
                    const float4 o = *reinterpret_cast<const float4 *>(p);
                    w.x = __float_as_uint(__uint_as_float(w.x) + o.x);
                    w.y = __float_as_uint(__uint_as_float(w.y) + o.y);
                    w.z = __float_as_uint(__uint_as_float(w.z) + o.z);
                    w.w = __float_as_uint(__uint_as_float(w.w) + o.w);
                }
                *p = w;
            }
        }
    } else {
        constexpr int kPer = 128 / ELEM;
#pragma unroll 4
        for (int e = lane; e < 32 * kPer; e += 32) {
            const int r = e / kPer, c = (e % kPer) * ELEM;
            if (r < rows && c < bytes) {
                char *p = out + (size_t)r * row_bytes + c;
                if (ELEM == 4) {
                    const float f = *reinterpret_cast<const float *>(stage + row_stage_at(r, c));
                    float *q = reinterpret_cast<float *>(p);
                    *q = accumulate ? *q + f : f;
                } else {
                    *reinterpret_cast<uint16_t *>(p) = *reinterpret_cast<const uint16_t *>(stage + row_stage_at(r, c));
                }
            }
        }
    }
    __syncwarp();
}

// ------------------------------------------------------------------------------ SwiGLU

// s(z) = 1 / (1 + e^-z).  The exponential and the division are CUDA's fast ones, documented as off by
// 2 + 1.2 |z| and 2 units in the last place (2^-23): for z > 0 the exponential's share of that shrinks
// with e^-z, for z < 0 s is off by (4 + 1.2 |z|) 2^-23 of its value, 2^-16 at z = -87.  The division is 0
// for divisors past 2^126, so s is 0 below z = -87.3 where its value is below 1.2e-38.  Both stay far
// below the rounding of the 16-bit results they feed (2^-12 of the value in fp16, 2^-9 in bf16).
__device__ __forceinline__ float sigmoid_f32(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
__device__ __forceinline__ float swiglu_value(float g, float u) { return g * sigmoid_f32(g) * u; }

// Gradients of h = silu(g) u: dg = dh u s (1 + g (1 - s)), du = dh g s.
__device__ __forceinline__ void swiglu_grads(float g, float u, float dh, float &dg, float &du) {
    const float s = sigmoid_f32(g);
    dg = dh * u * (s * fmaf(g, 1.f - s, 1.f));
    du = dh * (g * s);
}

// Tiles in groups of 8 row tiles by all column tiles, so that the pairs running at a time
// share both operands in L2.
__device__ __forceinline__ void grouped_tile(long long t, int m_tiles, int n_tiles, int &m, int &n) {
    const long long per = 8LL * n_tiles;
    const int g = (int)(t / per), r = (int)(t % per);
    const int rows = min(8, m_tiles - g * 8);
    m = g * 8 + r % rows;
    n = r / rows;
}

// ------------------------------------------------------------------------------ host

// Lets a kernel use `bytes` of dynamic shared memory on the current device, and loads it.
template <typename... KArgs>
static bool set_smem(void (*kernel)(KArgs...), int bytes) {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kernel) != cudaSuccess ||
           (bytes > 0 &&
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess);
}

// Largest size the tile arithmetic takes (sizes are rounded up to tiles in 32 bits).
constexpr int kMostSize = 0x7FFFFFFF - 1023;

// Tensor map of a row-major [rows][cols] matrix (rows packed) read in boxes of
// box_rows x one 128-byte row segment, 128-byte swizzle, zeros outside the matrix.
static int matrix_map(CUtensorMap *map, CUtensorMapDataType type, size_t esize, const void *base, long long rows,
                      long long cols, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return record_error("cuTensorMapEncodeTiled entry point not found");
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols * esize};
    cuuint32_t box[2] = {(cuuint32_t)(128 / esize), (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, type, 2, (void *)base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? TQ_OK : record_error("cuTensorMapEncodeTiled failed");
}

template <typename... KArgs, typename... Args>
inline cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                  int cluster, bool chained, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (chained) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace tq
