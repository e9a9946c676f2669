// Gated feed-forward block (SwiGLU) of a dense expert and its gradient.
//
//   g = x Wg^T, u = x Wu^T, h = silu(g) * u
//   dg = dh u s (1 + g (1 - s)), du = dh g s   (s = 1 / (1 + e^-g))
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
//
// Three products, all by one persistent CTA-pair kernel (tcgen05, cta_group::2): a pair
// owns a 256 x 256 tile of fp32 accumulators, each CTA its 128 rows in its own tensor
// memory (two tiles of 256 columns: the epilogue of one tile runs under the MMAs of the
// next).  Per K-block of 64 each CTA brings in its half of both operands (2 x 16 KB, 6
// stages) by TMA; the leader's MMA thread issues 4 MMAs of 256 x 256 x 16.
//   * What bounds it is those copies (about 45 B a clock and SM where a tile needs 62 at the
//     full MMA rate), and over many calls the power limit.  Where there are tiles enough, a pair
//     takes two neighbours at a time (WIDE: 256 x 512, both accumulators, 3 x 16 KB in 4 stages),
//     which reads A once for both.  Their epilogues then lie between the pairs of tiles,
//     except that the first half of the next may start while the second half of the last is
//     read out.  In a loop: forward 8192, 4096 -> 1024 113 us (119 without), its gradient 336
//     (350), forward 3000, 3000 -> 3000 78 (89, which also has the rounds in its favour).
//   * gate/up: the B operand's first half is 128 gate rows (CTA 0), its second half the
//     same 128 up rows (CTA 1), so a row's g and u meet in one thread's epilogue, which
//     writes h, or (backward) reads dh and writes dg and du.  128 columns are also one
//     scale block: the thread that holds a row of it stores g and u in 8 bits.
//   * gradients: one launch takes the tiles of dWg and dWu (both operands MN-major: K runs
//     over the tokens) and then those of dx (A K-major, B MN-major; K runs over Wg's rows
//     and then Wu's), so the long weight-gradient tiles start first and the dx tiles fill
//     the pairs that finish early.
// dg and du are rounded to bf16 between the two launches, because the tensor cores take 16-bit
// operands: at most 2^-8 of each term, and as the terms' errors are independent about as much
// of a sum as the rounding of the 16-bit gradient itself.  Measured against 64 bits, at every size:
// 0.0022-0.0026 of the gradients' norm, 0.0014-0.0018 for the last rounding alone.  That alone remains of
// a weight gradient with a second bf16 word for the remainder, that K then runs over too.  From
// 8-bit activations small problems have it, where dw tiles wait for dx tiles anyway (second_words);
// elsewhere it would cost up to half of the pass (from x its second pass over the tile 5.5 us: 512 tokens, 512
// -> 512 16.5 -> 22.1 us; from 8-bit activations 1064 tokens, 1000 -> 504 16.2 -> 24.6; 8192, 4096 -> 1024 209 ->
// 307).
//
// Few tokens: dense_rows_kernel (weights streamed once, tokens on the MMA's N side).
#include "tq_dense_rows.cuh"

#include <algorithm>

namespace tq {

constexpr int kPairM = 256, kPairN = 256;
constexpr int kPairRing = 192 * 1024;   // operand stages: 6 of 32 KB, or 4 of 48 KB (wide tiles)
constexpr int kPairStages = 6;
constexpr int kPairThreads = 384;      // warp 0 TMA, 1 MMA (leader), 2 TMEM, 4-11 epilogue
constexpr int kPairStageBytes = 16384;

struct __align__(1024) PairSmem {
    unsigned char ring[kPairRing];  // a stage: A, B, and in a wide tile the B of its second half
    unsigned char rows[8][kRowStage];
    uint64_t full[kPairStages];     // leader: both CTAs' copies of the stage
    uint64_t empty[kPairStages];    // MMA commit, in both CTAs
    uint64_t acc_full[2];           // MMA commit, in both CTAs
    uint64_t acc_empty[2];          // leader: the 16 epilogue warps of the pair
    uint32_t tmem_base;
    int32_t abort;
};
static_assert(sizeof(PairSmem) + 1024 <= 227 * 1024, "pair GEMM shared memory");

// gate/up: a0 = x, b0 = Wg, b1 = Wu.  Gradients: a0 = dg, a1 = du, b0 = Wg, b1 = Wu, x = x.
// Every map reads boxes of 64 x 64 elements.
struct PairMaps {
    CUtensorMap a0, a1, b0, b1, x;
    CUtensorMap a0_lo, a1_lo;     // weight gradients in two words: the second words of dg and du
};

struct PairArgs {
    int T, D, F;
    int f16;                                  // 16-bit type: 1 fp16, 0 bf16
    void *h;                                  // [T][F]
    uint8_t *g8, *u8;                         // [T][F] E4M3, or null
    float *sg, *su;                           // [T][ceil(F / 128)]
    const __nv_bfloat16 *dh;                  // [T][F]
    __nv_bfloat16 *dg, *du;                   // [T][F]
    int words;                                // of dg and du in the weight gradients: 1, 2
    __nv_bfloat16 *dx, *dwg, *dwu;            // [T][D], [F][D], [F][D]
    // tile plan (plan_gateup, plan_grads)
    int wide;                                 // tiles of 512 columns, counted as two of 256 each
    long long full;                           // gate/up: whole tiles; the others are halved
    long long tiles;                          // gate/up: tiles, halves counted one by one
    int halved;                               // gradients: every tile is half as wide
    int split_dw, split_dx;                   // gradients: pieces that K of a tile is cut into
    long long n_dw, n_dx;                     // gradients: pieces of each kind
    int more;                                 // gradients: pairs that have one dw piece more than the rest,
    long long dx_more, dx_rest;               //   and the dx pieces of such a pair and of another
    float *part_dw, *part_dx;                 // split: fp32 partial sums [piece][2 F][D], [piece][T][D]
};

enum PairKind { kPairForward = 0, kPairSave = 1, kPairRecompute = 2, kPairGrads = 3 };

// One output tile: rows m0 .. m0 + 255 of the pair, columns n0 .. n0 + width - 1 (gate/up:
// width / 2 outputs; width 256, or 128 for a halved tile), `which` the matrix of a weight
// gradient (0 gate, 1 up; -1 dx).  With K split it is one piece of a tile.
struct PairTile {
    int m0, n0, width, kblocks, which;
    int k0, part;      // gradients: first K-block, and which piece of K
};

// The j-th tile of a pair; false past its last.
template <int KIND, bool WIDE>
__device__ __forceinline__ bool pair_tile(const PairArgs &p, long long pair, long long pairs, long long j, PairTile &r) {
    int m, n;
    if (KIND != kPairGrads) {
        if (WIDE) {
            const long long t = pair + (j >> 1) * pairs;
            if (t >= p.tiles) return false;
            grouped_tile(t, (p.T + kPairM - 1) / kPairM, (p.F + 255) / 256, m, n);
            r.m0 = m * kPairM;
            r.n0 = n * 256 + 128 * (int)(j & 1);
            r.width = 256;
            r.kblocks = (p.D + 63) / 64;
            r.which = -1;
            r.k0 = r.part = 0;
            return true;
        }
        // whole tiles first, then the halves of the last ones
        long long t = pair + j * pairs;
        if (t >= p.tiles) return false;
        const bool half = t >= p.full;
        const int part = half ? (int)((t - p.full) & 1) : 0;
        if (half) t = p.full + ((t - p.full) >> 1);
        grouped_tile(t, (p.T + kPairM - 1) / kPairM, (p.F + 127) / 128, m, n);
        r.m0 = m * kPairM;
        r.n0 = n * 128 + 64 * part;
        r.width = half ? 128 : 256;
        r.kblocks = (p.D + 63) / 64;
        r.which = -1;
        r.k0 = r.part = 0;
        return true;
    }
    const int width = WIDE ? 512 : p.halved ? 128 : 256, second = WIDE ? (int)(j & 1) : 0;
    if (WIDE) j >>= 1;
    const int nd = (p.D + width - 1) / width, mf = (p.F + kPairM - 1) / kPairM;
    const bool more = pair < p.more;
    const long long dw = p.n_dw / pairs + (more ? 1 : 0);
    long long t;
    int k, split;
    if (j < dw) {
        t = pair + j * pairs;
        const long long tiles = 2LL * mf * nd;
        split = p.split_dw;
        r.part = (int)(t / tiles);
        grouped_tile(t % tiles, 2 * mf, nd, m, n);
        r.which = m >= mf;
        r.m0 = (m - (r.which ? mf : 0)) * kPairM;
        k = p.words * ((p.T + 63) / 64);
    } else {
        const long long i = j - dw, cut = p.more * p.dx_more;
        t = more ? pair + i * p.more : cut + (pair - p.more) + i * (pairs - p.more);
        if (i >= (more ? p.dx_more : p.dx_rest) || t >= p.n_dx) return false;
        const int mt = (p.T + kPairM - 1) / kPairM;
        const long long tiles = (long long)mt * nd;
        split = p.split_dx;
        r.part = (int)(t / tiles);
        grouped_tile(t % tiles, mt, nd, m, n);
        r.which = -1;
        r.m0 = m * kPairM;
        k = 2 * ((p.F + 63) / 64);
    }
    r.width = p.halved ? 128 : 256;
    r.n0 = n * width + 256 * second;
    r.k0 = (int)((long long)k * r.part / split);
    r.kblocks = (int)((long long)k * (r.part + 1) / split) - r.k0;
    return true;
}

// ------------------------------------------------------------------------------ epilogues

// 32 fp32 values of a row as 64 bytes of 16-bit values.
__device__ __forceinline__ void pack_row32(const float (&v)[32], bool f16, uint4 *p) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        p[j] = make_uint4(pack16(v[8 * j], v[8 * j + 1], f16), pack16(v[8 * j + 2], v[8 * j + 3], f16),
                          pack16(v[8 * j + 4], v[8 * j + 5], f16), pack16(v[8 * j + 6], v[8 * j + 7], f16));
}

// What rounding a value to bf16 leaves; 0 where that is no number (the first word says it then).
__device__ __forceinline__ float bf16_remainder(float v) {
    const float d = v - __bfloat162float(__float2bfloat16_rn(v));
    return fabsf(d) <= FLT_MAX ? d : 0.f;
}

// The h tile, or (GRADS) the dg and du tiles, of one warp: columns c0 .. c0 + 63 of its rows, or 32 of a
// halved tile (the second half of o is then not stored).
template <bool GRADS>
__device__ __forceinline__ void store_outputs(const PairArgs &p, const PairTile &t, uint32_t taddr, int r0, int lane,
                                              int w, unsigned char *stage) {
    uint32_t a[32], b[32];
    float v[32];
    uint4 o[8], o2[8];
    const bool halved = t.width != 256;
    const int c0 = (halved ? 32 : 64) * w, u0 = t.width / 2;
    const int r = r0 + lane, rows = p.T - r0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (half && halved) break;
        const int c = c0 + 32 * half;
        tmem_ld32(taddr + c, a);
        tmem_ld32(taddr + u0 + c, b);
        const int col = t.n0 + c;
        if constexpr (GRADS) {
            uint4 d[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                d[j] = r < p.T && col + 8 * j < p.F
                           ? *reinterpret_cast<const uint4 *>(p.dh + (size_t)r * p.F + col + 8 * j)
                           : make_uint4(0, 0, 0, 0);
            tmem_ld_wait();
            float du[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const uint32_t w2 = reinterpret_cast<const uint32_t *>(d)[i >> 1];
                const float dh = __uint_as_float((i & 1) ? (w2 & 0xFFFF0000u) : (w2 << 16));
                swiglu_grads(__uint_as_float(a[i]), __uint_as_float(b[i]), dh, v[i], du[i]);
            }
            pack_row32(v, false, o + 4 * half);
            pack_row32(du, false, o2 + 4 * half);
        } else {
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = swiglu_value(__uint_as_float(a[i]), __uint_as_float(b[i]));
            pack_row32(v, p.f16 != 0, o + 4 * half);
        }
    }
    const int col = t.n0 + c0;
    const int bytes = min((p.F - col) * 2, halved ? 64 : 128);
    const size_t at = (size_t)r0 * p.F + col;
    if constexpr (GRADS) {
        warp_store_rows<2>(stage, lane, o, reinterpret_cast<char *>(p.dg + at), (size_t)p.F * 2, rows, bytes, true);
        warp_store_rows<2>(stage, lane, o2, reinterpret_cast<char *>(p.du + at), (size_t)p.F * 2, rows, bytes, true);
    } else {
        warp_store_rows<2>(stage, lane, o, reinterpret_cast<char *>(p.h) + at * 2, (size_t)p.F * 2, rows, bytes, true);
    }
}

// One warp's share of a tile: rows row0 .. row0 + 31 of the tile (tensor-memory lane quarter
// taddr), column half w.  `stage`: the warp's row stage.
template <int KIND>
__device__ __forceinline__ void pair_epilogue(const PairArgs &p, const PairTile &t, uint32_t taddr, int row0, int lane,
                                              int w, unsigned char *stage) {
    if (t.n0 >= (KIND == kPairGrads ? p.D : p.F)) return;     // a wide tile's second half past the matrix
    uint32_t a[32], b[32];
    float v[32];
    uint4 o[8];
    const int r0 = t.m0 + row0;
    if constexpr (KIND == kPairGrads) {
        __nv_bfloat16 *out = t.which < 0 ? p.dx : (t.which ? p.dwu : p.dwg);
        const int rows = (t.which < 0 ? p.T : p.F) - r0;
        const int cols = t.width / 2;
        float *part = t.which < 0 ? p.part_dx : p.part_dw;     // null: K is not split
        if (part)
            part += (t.which < 0 ? (size_t)t.part * p.T + r0 : ((size_t)t.part * 2 + t.which) * p.F + r0) * p.D;
#pragma unroll 1
        for (int c = cols * w; c < cols * w + cols; c += 64) {
            tmem_ld32(taddr + c, a);
            tmem_ld32(taddr + c + 32, b);
            tmem_ld_wait();
            if (part) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[i] = half ? make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3])
                                    : make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
                    const int col = t.n0 + c + 32 * half;
                    warp_store_rows<4>(stage, lane, o, reinterpret_cast<char *>(part + col), (size_t)p.D * 4, rows,
                                       (p.D - col) * 4, true);
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(a[i]);
            pack_row32(v, false, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(b[i]);
            pack_row32(v, false, o + 4);
            const int col = t.n0 + c;
            warp_store_rows<2>(stage, lane, o, reinterpret_cast<char *>(out + (size_t)r0 * p.D + col), (size_t)p.D * 2,
                               rows, (p.D - col) * 2, true);
        }
        return;
    }
    const int r = r0 + lane, rows = p.T - r0;
    if constexpr (KIND == kPairSave) {
        // column half w stores matrix w (0: g, 1: u) of the 128-wide block in 8 bits
        const uint32_t m_addr = taddr + 128 * w;
        float m = 0.f;
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
            tmem_ld32(m_addr + c, a);
            tmem_ld32(m_addr + c + 32, b);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)     // columns past F hold zeros
                m = finite_max(finite_max(m, __uint_as_float(a[i])), __uint_as_float(b[i]));
        }
        const int e = e4m3_block_exponent(m);
        const float inv = exp2_int(-e);
        const int fb = (p.F + 127) / 128;
        if (r < p.T) (w ? p.su : p.sg)[(size_t)r * fb + t.n0 / 128] = exp2_int(e);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
            tmem_ld32(m_addr + c, a);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
                uint32_t q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    q[j] = e4m3x4_scaled(__uint_as_float(a[i + 4 * j]), __uint_as_float(a[i + 4 * j + 1]),
                                         __uint_as_float(a[i + 4 * j + 2]), __uint_as_float(a[i + 4 * j + 3]), inv);
                o[(c + i) / 16] = make_uint4(q[0], q[1], q[2], q[3]);
            }
        }
        // F % 16 == 8: rows are 8-byte aligned, stored in 2-byte pieces
        warp_store_rows<2>(stage, lane, o, reinterpret_cast<char *>((w ? p.u8 : p.g8) + (size_t)r0 * p.F + t.n0),
                           (size_t)p.F, rows, p.F - t.n0, p.F % 16 == 0);
    }
    store_outputs<KIND == kPairRecompute>(p, t, taddr, r0, lane, w, stage);
}

// ------------------------------------------------------------------------------ kernel

template <int KIND, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_gemm_kernel(const __grid_constant__ PairMaps maps, const PairArgs args) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    PairSmem &sm = *reinterpret_cast<PairSmem *>(smem_raw + pad);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const long long pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
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

    constexpr bool wide = WIDE;
    constexpr uint32_t stages = wide ? 4 : 6, stage_bytes = (wide ? 3 : 2) * kPairStageBytes;
    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            uint32_t s = 0, turn = 0, it = 0;         // stage, and how often the ring was filled
            // operand tile of 64 or 128 rows x 64 K in 64 x 64 boxes: K-major (rows then K)
            // or MN-major (K rows of 64 consecutive matrix columns)
            auto load = [&](unsigned char *dst, const CUtensorMap *m, int r0, int k0, bool mn, bool two, uint32_t bar) {
                tma_load_2d_pair(dst, m, mn ? r0 : k0, mn ? k0 : r0, bar);
                if (two) tma_load_2d_pair(dst + 8192, m, mn ? r0 + 64 : k0, mn ? k0 : r0 + 64, bar);
            };
            PairTile tl;
            for (long long j = 0; ok && pair_tile<KIND, WIDE>(args, pair, pairs, j, tl); j += 1 + wide) {
                const bool two = tl.width == 256;         // B rows of a CTA: 128, or 64
                const int nb = tl.n0 + (tl.width / 2) * rank;
                const uint32_t bytes =
                    2 * (wide ? 3 * kPairStageBytes : kPairStageBytes + (two ? kPairStageBytes : kPairStageBytes / 2));
                // dx: K-blocks of dg, then of du; dw: of the tokens, then again for the second word
                const int half = (args.F + 63) / 64, tokens = (args.T + 63) / 64;
                for (int kb = tl.k0; kb < tl.k0 + tl.kblocks; ++kb, ++it) {
                    if (turn > 0 && !wait(&sm.empty[s], (turn - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    unsigned char *a = sm.ring + s * stage_bytes, *b = a + kPairStageBytes, *b2 = b + kPairStageBytes;
                    const uint32_t bar = map_to_rank(smem_u32(&sm.full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], bytes);
                    const int ar = tl.m0 + 128 * rank;
                    if (KIND != kPairGrads) {
                        const CUtensorMap *w = rank ? &maps.b1 : &maps.b0;
                        load(a, &maps.a0, ar, kb * 64, false, true, bar);
                        load(b, w, tl.n0, kb * 64, false, two, bar);
                        if (wide) load(b2, w, tl.n0 + 128, kb * 64, false, true, bar);
                    } else if (tl.which >= 0) {
                        const bool lo = kb >= tokens;
                        const int k0 = (lo ? kb - tokens : kb) * 64;
                        load(a, tl.which ? (lo ? &maps.a1_lo : &maps.a1) : (lo ? &maps.a0_lo : &maps.a0), ar, k0, true,
                             true, bar);
                        load(b, &maps.x, nb, k0, true, two, bar);
                        if (wide) load(b2, &maps.x, nb + 256, k0, true, true, bar);
                    } else {
                        const bool up = kb >= half;
                        const int k0 = (up ? kb - half : kb) * 64;
                        const CUtensorMap *w = up ? &maps.b1 : &maps.b0;
                        load(a, up ? &maps.a1 : &maps.a0, ar, k0, false, true, bar);
                        load(b, w, nb, k0, true, two, bar);
                        if (wide) load(b2, w, nb + 256, k0, true, true, bar);
                    }
                    if (++s == stages) {
                        s = 0;
                        ++turn;
                    }
                }
            }
            // every stage read by its MMAs before the CTA can exit; after a wait that gave
            // up, time for the copies in flight to land
            for (uint32_t i = it > stages ? it - stages : 0; i < it && ok; ++i)
                ok = wait(&sm.empty[i % stages], (i / stages) & 1);
            if (!ok)
                for (int i = 0; i < 2000; ++i) __nanosleep(1000);
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            bool ok = true;
            uint32_t s = 0, turn = 0;
            const int fmt = args.f16 ? 0 : 1;
            PairTile tl;
            for (uint32_t j = 0; ok && pair_tile<KIND, WIDE>(args, pair, pairs, j, tl); j += 1 + wide) {
                const bool a_mn = KIND == kPairGrads && tl.which >= 0, b_mn = KIND == kPairGrads;
                const uint32_t idesc = umma_idesc(kPairM, tl.width, fmt, a_mn, b_mn);
                const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;   // 16-byte units per K = 16
                const uint32_t st = j & 1, parity = ((j >> 1) - 1) & 1;
                // MMAs of stage `at` into accumulator `acc`, from its B or (second) the wide tile's other
                auto multiply = [&](uint32_t at, uint32_t acc, bool second, bool first_block) {
                    const uint32_t as = smem_u32(sm.ring) + at * stage_bytes;
                    const uint32_t bs = as + (second ? 2 : 1) * kPairStageBytes;
                    const uint64_t ad = a_mn ? umma_desc_mn_sw128(as) : umma_desc_sw128(as);
                    const uint64_t bd = b_mn ? umma_desc_mn_sw128(bs) : umma_desc_sw128(bs);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f16_pair(tmem + acc * kPairN, ad + k * a_step, bd + k * b_step, idesc, !first_block || k != 0);
                };
                if (j >= 2 && !wait(&sm.acc_empty[st], parity)) break;
                // A wide tile's second half may follow the first by the ring: its accumulator is
                // still being read out when the first one is free.
                bool other = !wide || j < 2;
                int k2 = 0;                   // wide: next K-block of the second half, and its stage
                uint32_t s2 = s;
                tc_fence_after();
                for (int kb = 0; kb < tl.kblocks; ++kb) {
                    if (!wait(&sm.full[s], turn & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    multiply(s, st, false, kb == 0);
                    if (!wide) {
                        umma_commit_pair(&sm.empty[s]);
                    } else {
                        const bool last = kb + 1 == tl.kblocks;
                        if (last) umma_commit_pair(&sm.acc_full[st]);
                        if (!other) {
                            other = mbar_test(&sm.acc_empty[st ^ 1], parity);
                            if (!other && (last || kb + 1 - k2 == (int)stages)) {
                                if (!wait(&sm.acc_empty[st ^ 1], parity)) {
                                    ok = false;
                                    break;
                                }
                                other = true;
                            }
                            if (other) tc_fence_after();
                        }
                        for (; other && k2 <= kb; ++k2) {
                            multiply(s2, st ^ 1, true, k2 == 0);
                            umma_commit_pair(&sm.empty[s2]);
                            if (++s2 == stages) s2 = 0;
                        }
                    }
                    if (++s == stages) {
                        s = 0;
                        ++turn;
                    }
                }
                if (ok) umma_commit_pair(&sm.acc_full[wide ? st ^ 1 : st]);
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3, w = (warp - 4) >> 2;
        PairTile tl;
        for (uint32_t j = 0; pair_tile<KIND, WIDE>(args, pair, pairs, j, tl); ++j) {
            const uint32_t st = j & 1;
            const bool ok = __all_sync(0xffffffffu, wait(&sm.acc_full[st], (j >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            pair_epilogue<KIND>(args, tl, tmem + st * kPairN + ((uint32_t)(32 * q) << 16), 128 * rank + 32 * q, lane, w,
                                sm.rows[warp - 4]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(map_to_rank(smem_u32(&sm.acc_empty[st]), 0));
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

// Partial sums of gradients whose K was split, added in the pieces' order and rounded once: 8
// values a thread.  Memory-bound.
__global__ void __launch_bounds__(256) grads_reduce_kernel(const PairArgs p) {
    chain_entry();
    const long long nw = p.part_dw ? 2LL * p.F * p.D : 0, nx = p.part_dx ? (long long)p.T * p.D : 0;
    for (long long i = (blockIdx.x * 256LL + threadIdx.x) * 8; i < nw + nx; i += gridDim.x * 2048LL) {
        const bool w = i < nw;
        const long long at = w ? i : i - nw, n = w ? nw : nx;
        const float *src = (w ? p.part_dw : p.part_dx) + at;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const int pieces = w ? p.split_dw : p.split_dx;
#pragma unroll 4
        for (int k = 0; k < pieces; ++k) {
            float t[8];
            load8<float>(src + k * n, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += t[j];
        }
        const long long fd = (long long)p.F * p.D;
        __nv_bfloat16 *out = w ? (at < fd ? p.dwg + at : p.dwu + (at - fd)) : p.dx + at;
        *reinterpret_cast<uint4 *>(out) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
}

// What the gradients' products read, from the 8-bit activations, in one launch: the first
// blocks write x as bf16 (exact for scales that fp8_block_quantize made, down to bf16's least
// subnormal), the others dg and du.  Both take two rows of 512 columns a warp, as the 8-bit
// row kernels do.  Memory-bound.
struct SavedArgs {
    const uint8_t *x8, *g8, *u8;
    const float *sx, *sg, *su;
    const __nv_bfloat16 *dh;
    __nv_bfloat16 *x, *dg, *du, *dg_lo, *du_lo;     // second words: null with one
    int T, D, F;
    long long row_blocks, x_blocks;
};

__global__ void __launch_bounds__(kStoreWarps * 32) swiglu_saved_kernel(const SavedArgs p) {
    chain_entry();
    if (blockIdx.x < p.x_blocks) {
        fp8_dequantize_block(blockIdx.x % p.row_blocks, (int)(blockIdx.x / p.row_blocks), p.x8, p.sx, p.T, p.D, 1, p.x,
                             TQ_DTYPE_BF16);
        return;
    }
    const long long b = blockIdx.x - p.x_blocks;
    const int F = p.F, fb = (F + 127) / 128;
    const int r0 = (int)((b % p.row_blocks) * kStoreWarps + (threadIdx.x >> 5)) * kStoreRows;
    const int c0 = (int)(b / p.row_blocks) * 512 + (threadIdx.x & 31) * 8;
    uint2 gq[kStoreRows][2], uq[kStoreRows][2];
    uint4 d4[kStoreRows][2];
    float gs[kStoreRows][2], us[kStoreRows][2];
#pragma unroll
    for (int k = 0; k < kStoreRows; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int f = c0 + 256 * h;
            if (r0 + k >= p.T || f >= F) continue;
            const size_t at = (size_t)(r0 + k) * F + f, sat = (size_t)(r0 + k) * fb + f / 128;
            gq[k][h] = *reinterpret_cast<const uint2 *>(p.g8 + at);
            uq[k][h] = *reinterpret_cast<const uint2 *>(p.u8 + at);
            d4[k][h] = *reinterpret_cast<const uint4 *>(p.dh + at);
            gs[k][h] = p.sg[sat];
            us[k][h] = p.su[sat];
        }
#pragma unroll
    for (int k = 0; k < kStoreRows; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int f = c0 + 256 * h;
            if (r0 + k >= p.T || f >= F) continue;
            const size_t at = (size_t)(r0 + k) * F + f;
            float g[8], u[8], a[8], c[8];
            e4m3x4_to_f32(gq[k][h].x, *reinterpret_cast<float(*)[4]>(g));
            e4m3x4_to_f32(gq[k][h].y, *reinterpret_cast<float(*)[4]>(g + 4));
            e4m3x4_to_f32(uq[k][h].x, *reinterpret_cast<float(*)[4]>(u));
            e4m3x4_to_f32(uq[k][h].y, *reinterpret_cast<float(*)[4]>(u + 4));
            const uint32_t w[4] = {d4[k][h].x, d4[k][h].y, d4[k][h].z, d4[k][h].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
                swiglu_grads(g[j] * gs[k][h], u[j] * us[k][h], d, a[j], c[j]);
            }
            *reinterpret_cast<uint4 *>(p.dg + at) =
                make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7]));
            *reinterpret_cast<uint4 *>(p.du + at) =
                make_uint4(pack_bf16(c[0], c[1]), pack_bf16(c[2], c[3]), pack_bf16(c[4], c[5]), pack_bf16(c[6], c[7]));
            if (!p.dg_lo) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] = bf16_remainder(a[j]);
                c[j] = bf16_remainder(c[j]);
            }
            *reinterpret_cast<uint4 *>(p.dg_lo + at) =
                make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7]));
            *reinterpret_cast<uint4 *>(p.du_lo + at) =
                make_uint4(pack_bf16(c[0], c[1]), pack_bf16(c[2], c[3]), pack_bf16(c[4], c[5]), pack_bf16(c[6], c[7]));
        }
}

// ------------------------------------------------------------------------------ host side

static inline size_t align256_d(size_t n) { return (n + 255) & ~(size_t)255; }

// Estimated times of plan_grads in us: a K-block of 64 in a whole and a halved tile (whose MMAs take
// half as long; the copies' latency is the same), a piece's start and end, the launch that adds
// partial sums, and the bytes it moves in one.  Fitted by eye to the whole backward pass of ten shapes
// (64 to 8192 tokens, D and F of 256 to 4096) with each tile width and split forced in turn, on one B200:
// they rank plans.  As times they leave out what every plan has, the launch, the ring's filling and the
// last epilogue, and are about half of what a small problem takes (1111 tokens, 1000 -> 504: 11 of 21 us).
constexpr double kBlockUs = 0.35, kHalfBlockUs = 0.30, kWideBlockUs = 0.60, kPieceUs = 1.0, kWidePieceUs = 4.0,
                 kTileEndUs = 2.0, kReduceUs = 3.0, kReduceBytesUs = 4e6;

static int pair_map(CUtensorMap *m, const void *base, long long rows, long long cols, int f16) {
    return matrix_map(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, rows, cols,
                      64);
}

// Gate/up tiles, by estimated time: taken two at a time (8192 tokens, 4096 -> 1024: 128 double tiles,
// 2 rounds of 74 pairs, 113 us in a loop; 119 one by one), or one by one, where the tiles of a last round
// that leaves half of the pairs or more without work are halved in width (not where they store
// 8-bit blocks, which need all 128 columns; 1111 tokens, 1000 -> 504, 20 tiles as 40: the gradient's
// two launches 25.6 -> 20.6 us).
static long long plan_gateup(PairArgs &p, long long pairs, bool may_halve) {
    const long long mt = ((long long)p.T + kPairM - 1) / kPairM;
    const long long n = mt * ((p.F + 127LL) / 128), last = n % pairs, n2 = mt * ((p.F + 255LL) / 256);
    const bool halve = may_halve && 2 * last <= pairs;
    const double kb = (p.D + 63) / 64;
    const double t = std::max(kb * kBlockUs, kTileEndUs), t_half = std::max(kb * kHalfBlockUs, kTileEndUs);
    const double t_wide = std::max(kb * kWideBlockUs + 0.5 * kWidePieceUs, 2 * kTileEndUs);
    const double narrow = (double)(n / pairs) * t + (last == 0 ? 0 : halve ? t_half : t);
    p.wide = (double)((n2 + pairs - 1) / pairs) * t_wide < narrow;
    if (p.wide) return p.tiles = n2;
    p.full = halve ? n - last : n;
    p.tiles = p.full + 2 * (n - p.full);
    return p.tiles;
}

// Columns of a gradient tile: whole, halved, wide.
static long long grads_width(int mode) { return mode == 2 ? 512 : mode ? 128 : 256; }

// Deals the gradient pieces of one tile width and split to the pairs: the dw pieces (K over `words` bf16
// words of dg and du) go round the pairs first; the dx pieces then fill up, so that the most loaded
// pair has least.  Fills p's plan and returns that load (estimated us).
static double deal_grads(PairArgs &p, long long pairs, int mode, int s_dw, int s_dx, int words) {
    const long long mf = ((long long)p.F + kPairM - 1) / kPairM, mt = ((long long)p.T + kPairM - 1) / kPairM;
    const long long k_dw = words * (((long long)p.T + 63) / 64), k_dx = 2 * (((long long)p.F + 63) / 64);
    const long long nd = (p.D + grads_width(mode) - 1) / grads_width(mode);
    const double t_kb = mode == 2 ? kWideBlockUs : mode ? kHalfBlockUs : kBlockUs;
    const double t_piece = mode == 2 ? kWidePieceUs : kPieceUs;
    const long long n_dw = 2 * mf * nd * s_dw, n_dx = mt * nd * s_dx;
    const double u_dw = (double)((k_dw + s_dw - 1) / s_dw) * t_kb + t_piece;
    const double u_dx = (double)((k_dx + s_dx - 1) / s_dx) * t_kb + t_piece;
    const long long on = n_dw + n_dx < pairs ? n_dw + n_dx : pairs;      // pairs at work
    const long long q = n_dw / on, more = n_dw % on, rest = on - more;
    // dx pieces of a pair with q + 1 dw pieces: a, of the others: b.  Level loads are
    // at a = (n_dx u_dx / rest - u_dw) / (u_dx (1 + more / rest)); whole numbers next to it.
    long long a = 0, b = 0;
    double load = -1;
    const double level = (n_dx * u_dx / rest - u_dw) / (u_dx * (1.0 + (double)more / rest));
    const long long top = more ? (n_dx + more - 1) / more : 0, x0 = level > 1 ? (long long)level - 1 : 0;
    for (long long x = x0 < top ? x0 : top; x <= top && x <= x0 + 3; ++x) {
        const long long left = n_dx - more * x, y = left > 0 ? (left + rest - 1) / rest : 0;
        const double l1 = more ? (q + 1) * u_dw + x * u_dx : 0, l0 = q * u_dw + y * u_dx;
        const double l = l1 > l0 ? l1 : l0;
        if (load < 0 || l < load) {
            load = l;
            a = x;
            b = y;
        }
    }
    p.words = words;
    p.halved = mode == 1;
    p.wide = mode == 2;
    p.split_dw = s_dw;
    p.split_dx = s_dx;
    p.n_dw = n_dw;
    p.n_dx = n_dx;
    p.more = (int)more;
    p.dx_more = a;
    p.dx_rest = b;
    return load;
}

// Gradient tiles.  Where there are few they are halved in width, and K of either kind is split (dw:
// many tokens and a small weight; dx: few tokens and a large one): the pieces' fp32 sums are then
// added by one more launch.  The choice is the least of the estimated times.  Whole backward pass, GPU
// us, as chosen and in one whole piece a tile: 8192 tokens, 512 -> 256 26 (dw in 8 pieces), 56; 64
// tokens, 4096 -> 4096 59 (dx in 4), 85; 512 tokens, 2048 -> 2048 41 (dx in 4), 48; 1111 tokens, 1000 ->
// 504 22 (halved), 24.  The plan is one for one word of dg and du; returns its load.
static double plan_grads(PairArgs &p, long long pairs) {
    const long long mf = ((long long)p.F + kPairM - 1) / kPairM, mt = ((long long)p.T + kPairM - 1) / kPairM;
    const long long k_dw = ((long long)p.T + 63) / 64, k_dx = 2 * (((long long)p.F + 63) / 64);
    double best = -1, load = 0;
    PairArgs best_plan = p;
    for (int mode = 0; mode < 3; ++mode) {                 // whole, halved, wide
        const long long nd = (p.D + grads_width(mode) - 1) / grads_width(mode);
        for (int s_dw = 1; s_dw <= 16 && (s_dw == 1 || s_dw * 4 <= k_dw); s_dw *= 2)
            for (int s_dx = 1; s_dx <= 16 && (s_dx == 1 || s_dx * 4 <= k_dx); s_dx *= 2) {
                // a split is for few tiles: no more pieces than pairs
                if ((s_dw > 1 && 2 * mf * nd * s_dw > pairs) || (s_dx > 1 && mt * nd * s_dx > 2 * pairs)) break;
                const double l = deal_grads(p, pairs, mode, s_dw, s_dx, 1);
                const double sums = (s_dw > 1 ? 2.0 * s_dw * p.F * p.D : 0) + (s_dx > 1 ? 1.0 * s_dx * p.T * p.D : 0);
                const double cost = l + (sums > 0 ? kReduceUs + 8 * sums / kReduceBytesUs : 0);
                if (best < 0 || cost < best) {
                    best = cost;
                    load = l;
                    best_plan = p;
                }
            }
    }
    p = best_plan;
    return load;
}

// Whether a plan of that load has room for second words of dg and du: the launch with them ends no
// later, but for a K-block's time, counting the words' own bytes.  p then is the plan with them.
// Backward pass from 8-bit activations, GPU us, with them and, for a few tokens more, without: 512 -> 512
// 12.7 (512 tokens), 11.9 (520); 1000 -> 504 14.0 (504), 13.9 (520); 1032 -> 392 14.4 (384), 12.7 (450).
static bool second_words(PairArgs &p, long long pairs, double load) {
    PairArgs two = p;
    const double l = deal_grads(two, pairs, p.wide ? 2 : p.halved, p.split_dw, p.split_dx, 2);
    if (l + 4.0 * p.T * p.F / kReduceBytesUs > load + kBlockUs) return false;
    p = two;
    return true;
}

// fp32 partial sums of the plan.
static size_t grads_part_bytes(const PairArgs &p, bool dx) {
    if (dx) return p.split_dx > 1 ? align256_d((size_t)p.split_dx * p.T * p.D * 4) : 0;
    return p.split_dw > 1 ? align256_d((size_t)p.split_dw * 2 * p.F * p.D * 4) : 0;
}

template <int KIND>
static int launch_pair(const PairMaps &maps, PairArgs p, cudaStream_t s, int stage) {
    const int smem = (int)sizeof(PairSmem) + 1024;
    const long long pairs = num_sms() / 2;
    const long long tiles = KIND == kPairGrads ? p.n_dw + p.n_dx : plan_gateup(p, pairs, KIND != kPairSave);
    const unsigned grid = 2 * (unsigned)(tiles < pairs ? tiles : pairs);
    LaunchScope ls(s, stage);
    auto kernel = p.wide ? pair_gemm_kernel<KIND, true> : pair_gemm_kernel<KIND, false>;
    if (launch_chained(kernel, dim3(grid), dim3(kPairThreads), smem, s, maps, p) != cudaSuccess)
        return record_cuda_error("pair_gemm_kernel");
    return launch_status();
}

template <int KIND>
static bool set_pair_smem() {
    const int smem = (int)sizeof(PairSmem) + 1024;
    return set_smem(pair_gemm_kernel<KIND, false>, smem) || set_smem(pair_gemm_kernel<KIND, true>, smem);
}

// The first call of an entry point on a device sets up every kernel that a later call of it may
// launch (their launch attributes; loading them), so that later calls may be captured.
static int configure_swiglu() {
    static PerDeviceFlag configured;
    if (configured.get()) return TQ_OK;
    if (set_pair_smem<kPairForward>() || set_pair_smem<kPairSave>() || set_pair_smem<kPairRecompute>() ||
        set_pair_smem<kPairGrads>() || configure_rows<16, kSwiglu>() ||
        configure_rows<32, kSwiglu>() || configure_rows<64, kSwiglu>() || configure_rows<128, kSwiglu>() ||
        set_smem(swiglu_saved_kernel, 0) || set_smem(grads_reduce_kernel, 0) || configure_store())
        return record_cuda_error("configure_swiglu");
    configured.set();
    return TQ_OK;
}

// Largest D and F.  Byte counts of a row's rest, (D - column) * 4, are 32-bit; a wait for an accumulator
// covers the whole of K, which at 0.6 us a K-block stays below a second here (a bounded wait gives up
// after four); and 65535 groups of 512 columns is what the 8-bit row kernels' grid holds.
constexpr int kMostFeatures = 65535 * 512;

static int swiglu_shape_status(int T, int D, int F) {
    if (T < 0 || D < 1 || F < 1 || D % 8 || F % 8) return TQ_ERR_INVALID_ARG;
    if (T > kMostSize || D > kMostFeatures || F > kMostFeatures) return TQ_ERR_UNSUPPORTED;
    return TQ_OK;
}

static bool saved_complete(const tq_swiglu_saved *s) { return s->x && s->s_x && s->g && s->s_g && s->u && s->s_u; }
static bool saved_aligned(const tq_swiglu_saved *s) {
    return aligned16(s->x) && aligned16(s->s_x) && aligned16(s->g) && aligned16(s->s_g) && aligned16(s->u) &&
           aligned16(s->s_u);
}

// Tokens the weight-streaming kernel takes: up to 128 (it is bound by reading the weights), and
// as many more as leave two CTAs a tile of 128 tokens by 64 outputs, two CTAs a SM: the pair
// kernel then has too few tiles (203 tokens, 2056 -> 1000: 8.7 us here, 14.3 there; 1024 tokens,
// 4096 -> 1024: 19.4 here, 24.4 there; 2048 tokens: 31.8 here, 26.3 there).
static bool swiglu_rows_case(int T, int F) {
    return T <= 128 || ((T + 127LL) / 128) * ((F + 63LL) / 64) <= num_sms();
}

static int swiglu_rows(const void *x, const void *wg, const void *wu, int f16, int T, int D, int F, void *h,
                       cudaStream_t s) {
    const CUtensorMapDataType ty = f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int n = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
    CUtensorMap mg, mu, mx;
    int st = matrix_map(&mg, ty, 2, wg, F, D, 64);
    if (!st) st = matrix_map(&mu, ty, 2, wu, F, D, 64);
    if (!st) st = matrix_map(&mx, ty, 2, x, T, D, n);
    if (st) return st;
    RowsArgs a{};
    a.rows = T;
    a.width = F;
    a.kblocks = (D + 63) / 64;
    a.out_type = f16 ? TQ_DTYPE_F16 : TQ_DTYPE_BF16;
    a.out = h;
    LaunchScope ls(s, kStageSwiglu);
    switch (n) {
        case 16: return launch_rows<16, kSwiglu>(mg, mu, mx, a, s, true);
        case 32: return launch_rows<32, kSwiglu>(mg, mu, mx, a, s, true);
        case 64: return launch_rows<64, kSwiglu>(mg, mu, mx, a, s, true);
        default: return launch_rows<128, kSwiglu>(mg, mu, mx, a, s, true);
    }
}

}  // namespace tq

TQ_API int swiglu_forward(const void *x, const void *w_gate, const void *w_up, int dtype, int T, int D, int F, void *h,
                          const tq_swiglu_saved *saved, tq_stream stream) {
    using namespace tq;
    if (dtype != TQ_DTYPE_F16 && dtype != TQ_DTYPE_BF16)
        return dtype == TQ_DTYPE_F32 ? TQ_ERR_UNSUPPORTED : TQ_ERR_INVALID_ARG;
    int st = swiglu_shape_status(T, D, F);
    if (st) return st;
    if (T == 0) return TQ_OK;
    if (!x || !w_gate || !w_up || !h || (saved && !saved_complete(saved))) return TQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(h) || (saved && !saved_aligned(saved)))
        return TQ_ERR_ALIGNMENT;
    if ((st = configure_swiglu())) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    const int f16 = dtype == TQ_DTYPE_F16;
    if (!saved && swiglu_rows_case(T, F)) return swiglu_rows(x, w_gate, w_up, f16, T, D, F, h, s);
    if (saved) {
        st = fp8_block_quantize(x, dtype, T, D, 1, saved->x, saved->s_x, stream);
        if (st) return st;
    }
    PairMaps maps;
    memset(&maps, 0, sizeof(maps));
    st = pair_map(&maps.a0, x, T, D, f16);
    if (!st) st = pair_map(&maps.b0, w_gate, F, D, f16);
    if (!st) st = pair_map(&maps.b1, w_up, F, D, f16);
    if (st) return st;
    PairArgs p{};
    p.T = T;
    p.D = D;
    p.F = F;
    p.f16 = f16;
    p.h = h;
    if (!saved) return launch_pair<kPairForward>(maps, p, s, kStageSwiglu);
    p.g8 = saved->g;
    p.u8 = saved->u;
    p.sg = saved->s_g;
    p.su = saved->s_u;
    return launch_pair<kPairSave>(maps, p, s, kStageSwiglu);
}

namespace tq {
// Workspace of a backward call whose plan p holds: dg, du (with second words where `two`), x as bf16
// (from_saved), partial sums.
static size_t backward_bytes(const PairArgs &p, bool two, bool from_saved) {
    return (two ? 4 : 2) * align256_d((size_t)p.T * p.F * 2) + (from_saved ? align256_d((size_t)p.T * p.D * 2) : 0) +
           grads_part_bytes(p, false) + grads_part_bytes(p, true);
}
}  // namespace tq

TQ_API size_t swiglu_backward_workspace_size(int T, int D, int F, int from_saved) {
    if (tq::swiglu_shape_status(T, D, F) || T == 0) return 0;
    tq::PairArgs p{};
    p.T = T;
    p.D = D;
    p.F = F;
    const long long pairs = tq::num_sms() / 2;
    const double load = tq::plan_grads(p, pairs);
    return tq::backward_bytes(p, tq::second_words(p, pairs, load), from_saved != 0);
}

TQ_API int swiglu_backward(const void *dh, const void *x, const tq_swiglu_saved *saved, const void *w_gate,
                           const void *w_up, int dtype, int T, int D, int F, void *dx, void *dw_gate, void *dw_up,
                           void *ws, size_t ws_bytes, tq_stream stream) {
    using namespace tq;
    if (dtype != TQ_DTYPE_BF16)
        return dtype == TQ_DTYPE_F16 || dtype == TQ_DTYPE_F32 ? TQ_ERR_UNSUPPORTED : TQ_ERR_INVALID_ARG;
    int st = swiglu_shape_status(T, D, F);
    if (st) return st;
    if (!dw_gate || !dw_up) return TQ_ERR_INVALID_ARG;
    if (!aligned16(dw_gate) || !aligned16(dw_up)) return TQ_ERR_ALIGNMENT;
    const cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {      // an empty batch: dx has no rows, the weight gradients are zero
        if (cudaMemsetAsync(dw_gate, 0, (size_t)F * D * 2, s) != cudaSuccess ||
            cudaMemsetAsync(dw_up, 0, (size_t)F * D * 2, s) != cudaSuccess)
            return record_cuda_error("swiglu_backward: memset");
        return TQ_OK;
    }
    if (!dh || !w_gate || !w_up || !dx || (x != nullptr) == (saved != nullptr)) return TQ_ERR_INVALID_ARG;
    if (saved && !saved_complete(saved)) return TQ_ERR_INVALID_ARG;
    if (!aligned16(dh) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(dx) || (x && !aligned16(x)) ||
        (saved && !saved_aligned(saved)) || (ws && !aligned16(ws)))
        return TQ_ERR_ALIGNMENT;
    PairArgs p{};
    p.T = T;
    p.D = D;
    p.F = F;
    const long long pairs = num_sms() / 2;
    const double load = plan_grads(p, pairs);
    // the workspace is one size for both forms but for x; only the one from 8-bit activations has
    // second words
    PairArgs two = p;
    const bool has_two = second_words(two, pairs, load);
    if (!ws || ws_bytes < backward_bytes(p, has_two, saved != nullptr)) return TQ_ERR_WORKSPACE;
    if (saved && has_two) p = two;

    if ((st = configure_swiglu())) return st;
    char *w = reinterpret_cast<char *>(ws);
    p.dh = reinterpret_cast<const __nv_bfloat16 *>(dh);
    p.dg = reinterpret_cast<__nv_bfloat16 *>(w);
    w += align256_d((size_t)T * F * 2);
    p.du = reinterpret_cast<__nv_bfloat16 *>(w);
    w += align256_d((size_t)T * F * 2);
    __nv_bfloat16 *dg_lo = nullptr, *du_lo = nullptr;
    if (p.words == 2) {
        dg_lo = reinterpret_cast<__nv_bfloat16 *>(w);
        w += align256_d((size_t)T * F * 2);
        du_lo = reinterpret_cast<__nv_bfloat16 *>(w);
        w += align256_d((size_t)T * F * 2);
    }
    p.dx = reinterpret_cast<__nv_bfloat16 *>(dx);
    p.dwg = reinterpret_cast<__nv_bfloat16 *>(dw_gate);
    p.dwu = reinterpret_cast<__nv_bfloat16 *>(dw_up);
    PairMaps maps;
    memset(&maps, 0, sizeof(maps));
    st = pair_map(&maps.b0, w_gate, F, D, 0);
    if (!st) st = pair_map(&maps.b1, w_up, F, D, 0);
    if (st) return st;
    const void *xb = x;
    void *x_bf16 = w;
    if (saved) w += align256_d((size_t)T * D * 2);
    if (p.split_dw > 1) p.part_dw = reinterpret_cast<float *>(w);
    w += grads_part_bytes(p, false);
    if (p.split_dx > 1) p.part_dx = reinterpret_cast<float *>(w);
    if (saved) {
        SavedArgs a{};
        a.x8 = saved->x;
        a.g8 = saved->g;
        a.u8 = saved->u;
        a.sx = saved->s_x;
        a.sg = saved->s_g;
        a.su = saved->s_u;
        a.dh = p.dh;
        a.x = reinterpret_cast<__nv_bfloat16 *>(x_bf16);
        a.dg = p.dg;
        a.du = p.du;
        a.dg_lo = dg_lo;
        a.du_lo = du_lo;
        a.T = T;
        a.D = D;
        a.F = F;
        const dim3 gx = store_grid(T, D), gf = store_grid(T, F);
        a.row_blocks = gx.x;
        a.x_blocks = (long long)gx.x * gx.y;
        const long long blocks = a.x_blocks + (long long)gf.x * gf.y;
        if (blocks > 0x7FFFFFFFLL) return TQ_ERR_UNSUPPORTED;
        xb = x_bf16;
        LaunchScope ls(s, kStageSwigluGrad);
        if (launch_chained(swiglu_saved_kernel, dim3((unsigned)blocks), dim3(kStoreWarps * 32), 0, s, a) != cudaSuccess)
            return record_cuda_error("swiglu_saved_kernel");
    } else {
        st = pair_map(&maps.a0, x, T, D, 0);
        if (st) return st;
        st = launch_pair<kPairRecompute>(maps, p, s, kStageSwigluGrad);
    }
    if (st) return st;
    st = pair_map(&maps.a0, p.dg, T, F, 0);
    if (!st) st = pair_map(&maps.a1, p.du, T, F, 0);
    if (!st) st = pair_map(&maps.x, xb, T, D, 0);
    if (!st && p.words == 2) st = pair_map(&maps.a0_lo, dg_lo, T, F, 0);
    if (!st && p.words == 2) st = pair_map(&maps.a1_lo, du_lo, T, F, 0);
    if (!st) st = launch_pair<kPairGrads>(maps, p, s, kStageSwigluGrad);
    if (st || (!p.part_dw && !p.part_dx)) return st;
    const long long n = (p.part_dw ? 2LL * F * D : 0) + (p.part_dx ? (long long)T * D : 0);
    const long long blocks = (n / 8 + 255) / 256, most = 8LL * num_sms();
    LaunchScope ls(s, kStageSwigluGrad);
    if (launch_chained(grads_reduce_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s, p) !=
        cudaSuccess)
        return record_cuda_error("grads_reduce_kernel");
    return launch_status();
}

TQ_API int swiglu_backward_plan(int T, int D, int F, int32_t *plan) {
    const int st = tq::swiglu_shape_status(T, D, F);
    if (st) return st;
    if (T == 0 || !plan) return TQ_ERR_INVALID_ARG;
    tq::PairArgs p{};
    p.T = T;
    p.D = D;
    p.F = F;
    const long long pairs = tq::num_sms() / 2;
    tq::plan_gateup(p, pairs, true);
    plan[4] = p.wide ? 512 : p.full < p.tiles ? 128 : 256;
    tq::second_words(p, pairs, tq::plan_grads(p, pairs));
    plan[0] = p.words;
    plan[1] = p.wide ? 512 : p.halved ? 128 : 256;
    plan[2] = p.split_dw;
    plan[3] = p.split_dx;
    return TQ_OK;
}
