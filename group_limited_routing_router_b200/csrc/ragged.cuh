// Matrix products grouped by expert over ragged rows, as operators of their own (the expert half of
// the layer fuses its two; these are for training and for callers that compose their own experts).
// Group e owns rows offsets[e] <= r < offsets[e + 1]:
//   forward   out[r, n] = sum_k x[r, k] w[e, n, k]
//   dgrad     dx[r, k]  = sum_n dy[r, n] w[e, n, k]
//   wgrad     dw[e, n, k] (+)= sum_{r in e} dy[r, n] x[r, k]
//   INT8      out[r, n] = (sum_k q[r, k] wq[e, n, k]) * row_scale[r] * channel_scale[e, n]
// bf16 / fp16 operands (one type per call; the MMA's type field is a run-time value) with FP32
// accumulation, or INT8 operands with exact INT32 accumulation.
//
// Forward and dgrad are swap-AB: the MMA's M side walks the output features (weight rows in the
// forward pass, weight columns in dgrad), its N side the group's rows, rounded up to 16 (INT8 pairs:
// 32), so a group of a few rows wastes little and a weight byte crosses HBM once per token tile.
// dgrad reads the same [E, N, K] weights: their tile is the MMA's MN-major A operand, so no
// transposed copy of the weights exists.  wgrad contracts over the rows: both operands are MN-major.
//
// Accumulation.  The tensor core truncates its FP32 running sum at each instruction, so long sums are cut into
// segments of `seg_kb` k-steps: each accumulates in its own TMEM slot, and the epilogue adds the segments in
// FP32 registers, to nearest, while the next one's products run in the other slot (segment_steps and
// one_segment_ok in ragged_api.cuh say how long they are and why).
//
// Every mbarrier wait is bounded (status word BEAM_MOE_ERR_DEVICE_TIMEOUT on expiry); offsets that do
// not ascend within [0, R] set BEAM_MOE_ERR_BAD_INDEX and nothing is written; no load uses multicast.
#pragma once

#include <cuda_fp16.h>

#include "gemm_2sm.cuh"
#include "gemm_mx8.cuh"
#include "launch.cuh"

namespace beam {

constexpr int kRgThreads = 320;       // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue (pairs)
constexpr int kRgOperand = 16384;     // one staged operand tile: 128 rows of 128 bytes
constexpr int kRgRowBytes = 128;      // contraction bytes per k-step (64 16-bit or 128 8-bit elements)

struct RaggedParams {
    const int64_t *offsets;      // [E + 1], or NULL: one group of all R rows
    void *out;
    int64_t ldo;                 // output row stride, elements (forward, dgrad)
    int64_t R;
    int E;
    int M;                       // output features (forward: N, dgrad: K)
    int n_kb;                    // k-steps of 128 bytes over the contraction
    int seg_kb;                  // k-steps per accumulation segment
    int out_type;                // BEAM_MOE_BF16 / F16 / F32
    uint32_t idesc;              // instruction descriptor without N
    const float *row_scale;      // INT8: [R]
    const float *channel_scale;  // INT8: [E, M]
    long long timeout;
};

// ---- tcgen05 pieces ------------------------------------------------------------------------------
// MN-major operand written by TMA with 128-byte swizzling: boxes of 64 MN elements (128 bytes) by 64
// contraction rows; 8-row groups are 1024 B apart (stride byte offset), the next 64 MN elements one
// box = 8192 B further (leading byte offset).  One instruction takes 16 contraction rows: 2048 B.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(8192u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Eight accumulator columns twice over (16 columns) of 16 of the warp's TMEM lanes, as 8 x 8 fragments: this
// thread gets lane t / 4 (r[4 j], r[4 j + 1]) and lane t / 4 + 8 (r[4 j + 2], r[4 j + 3]) of columns
// 8 j + 2 (t % 4) and the next.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
// Four 8 x 8 fragments of 16-bit values, each stored transposed: thread 8 m + i gives the address of row i (16
// bytes) of matrix m, which receives column i of fragment m.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ uint32_t idesc_with_n(uint32_t idesc, int n) {
    return idesc | (static_cast<uint32_t>(n >> 3) << 17);
}

// Arrives on a barrier of any CTA of the cluster without a release at cluster scope, which would wait for all of the
// thread's earlier memory operations.  What is handed over is TMEM, ordered by the tcgen05 fences on both sides.
__device__ __forceinline__ void mbar_arrive_async(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// The same behind a release at cluster scope of shared memory alone: what the warp has read there may be overwritten
// by whoever acquires it, and what it has written (and fenced for the async proxy) is seen.  wgrad, 256 groups of ~78
// rows, 512 x 512: 38 us as without any release, 49 with one of all memory (64 groups of 128 rows, 5120 x 2560: 389
// against 431).
__device__ __forceinline__ void mbar_release_smem(uint32_t bar_cluster) {
    asm volatile(
        "fence.release.sync_restrict::shared::cta.cluster;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
        : "memory");
}
// Its other side, behind the wait on the barrier (which acquires at CTA scope).
__device__ __forceinline__ void acquire_smem() {
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

// ---- groups --------------------------------------------------------------------------------------
__device__ __forceinline__ int64_t group_begin(const RaggedParams &p, int e) { return p.offsets ? p.offsets[e] : 0; }
__device__ __forceinline__ int group_rows(const RaggedParams &p, int e) {
    return static_cast<int>(p.offsets ? p.offsets[e + 1] - p.offsets[e] : p.R);
}

// Rows of a group's row tiles: as few tiles of at most BN rows as hold them, of even size (a 273-row group in
// tiles of 256 and 17 would stream its weights a second time for 17 rows).  ROUND is the MMA's step in N.
template <int BN, int ROUND>
__device__ __forceinline__ int tile_rows(int rows) {
    const int n_nt = max(1, (rows + BN - 1) / BN);
    return ((rows + n_nt - 1) / n_nt + ROUND - 1) / ROUND * ROUND;
}

// Exclusive prefix of the groups' item counts in tile_start[0..E]: n_mt items per row tile of a group (WGRAD:
// n_mt items per group, `skip_empty` leaving out groups without rows).  Offsets that do not ascend within
// [0, R] give no items at all.  Contains __syncthreads; E <= 256 <= blockDim.x.
template <int BN, bool WGRAD>
__device__ __forceinline__ void ragged_prefix(const RaggedParams &p, int n_mt, bool skip_empty, int *tile_start) {
    __shared__ int warp_tot[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = threadIdx.x;
    int v = 0, bad = 0;
    if (e < p.E) {
        const int64_t lo = p.offsets ? p.offsets[e] : 0, hi = p.offsets ? p.offsets[e + 1] : p.R;
        bad = lo < 0 || hi < lo || hi > p.R;
        const int64_t rows = bad ? 0 : hi - lo;
        if (WGRAD) v = (skip_empty && rows == 0) ? 0 : n_mt;
        else v = n_mt * static_cast<int>((rows + BN - 1) / BN);
    }
    bad = __syncthreads_or(bad);
    if (bad) v = 0;
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) set_status(BEAM_MOE_ERR_BAD_INDEX);
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += warp_tot[w];
    if (e < p.E) tile_start[e] = base + incl - v;
    if (e == p.E - 1) tile_start[p.E] = base + incl;
}

__device__ __forceinline__ int find_group(int item, const int *tile_start, int E) {
    int lo = 0, hi = E - 1;  // largest e with tile_start[e] <= item
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tile_start[mid] <= item) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Forward / dgrad item: feature tile mt, row tile of group e.  The items a role decodes ascend: `e` starts at
// the first one's group (find_group) and walks along.
struct RaggedItem {
    int e, mt, n_valid, n_mma;
    int once;  // the group has one row tile, so its weights are read once: L2 evict-first
    int64_t row0;
};
// Bands of 8 row tiles go over all feature tiles in turn, so that what runs at one time reads some 8 row tiles and
// 9 feature tiles of 256; with all row tiles of a feature tile first it is 75 tiles, and the rows of a long group
// come from HBM for each feature tile (bf16, NA = 1: 16384 rows, 5120 x 2048, 271 -> 237 us; 32768 rows, 2048 x
// 4096, 418 -> 354; bands of 4 and 16 measure alike, of 32 1 to 3% more).
constexpr int kBandTiles = 8;
template <int BN, int ROUND>
__device__ __forceinline__ RaggedItem ragged_item(int item, int &e, int n_mt, const int *tile_start,
                                                  const RaggedParams &p) {
    RaggedItem it;
    while (tile_start[e + 1] <= item) ++e;
    it.e = e;
    const int rows = group_rows(p, e);
    const int n_nt = (rows + BN - 1) / BN;
    const int per = n_nt == 1 ? (rows + ROUND - 1) / ROUND * ROUND : tile_rows<BN, ROUND>(rows);
    const int local = item - tile_start[e];
    int nt = 0;
    it.mt = local;
    if (n_nt > 1) {
        const int band = local / (kBandTiles * n_mt), left = local - band * kBandTiles * n_mt;
        const int tiles = min(kBandTiles, n_nt - band * kBandTiles);
        it.mt = left / tiles;
        nt = band * kBandTiles + left - it.mt * tiles;
    }
    it.n_valid = min(per, rows - nt * per);  // > 0: rows > BN (n_nt - 1) >= per (n_nt - 1)
    it.n_mma = (it.n_valid + ROUND - 1) / ROUND * ROUND;
    it.once = n_nt == 1;
    it.row0 = group_begin(p, it.e) + static_cast<int64_t>(nt) * per;
    return it;
}

// ---- output ----------------------------------------------------------------------------------------
// Two values to a pair of 16-bit floats, nearest even.
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (TYPE == BEAM_MOE_F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// The epilogue's value of an accumulator: INT8 sums take their channel's and then their row's scale in FP32 (in
// this order the product of a large sum and a small scale comes first, and no product of two small ones).
template <bool I8>
__device__ __forceinline__ float ragged_value(uint32_t acc, float channel, float row) {
    return I8 ? static_cast<float>(static_cast<int32_t>(acc)) * channel * row : __uint_as_float(acc);
}

// fp32 results: feature m (this lane) of rows c .. c + 15, 128 bytes per row and warp.
__device__ __forceinline__ void store_cols(const RaggedParams &p, const RaggedItem &it, int c, int m,
                                           const float (&v)[16]) {
    float *o = reinterpret_cast<float *>(p.out) + (it.row0 + c) * p.ldo + m;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        if (c + j < it.n_valid && m < p.M) o[j * p.ldo] = v[j];
}

// 16-bit results.  The accumulators come as 8 x 8 fragments (tmem_ld_frag for lanes 0..15, then 16..31 of the
// warp), are packed in pairs of rows, and are turned by a transposing matrix store into [row][feature] order in a
// staging buffer that the four warps of a chunk's 128 features share, so that each store instruction covers two
// whole rows of 256 bytes.  45231 rows, 224 x 4328: 141 us (filling the result alone takes 100 to 120); 219 with
// 64 bytes per row and warp, 241 with pairs exchanged between lanes and 4 bytes stored per lane.
constexpr int kStage16 = 4096;  // a staging buffer: 16 rows x 128 features
constexpr int kStage16All = 4 * kStage16;  // two per group of four warps

// The four epilogue warps that share a chunk (`sub` 0 or 1).  They run the same chunks of the same items, after a
// wait that has timed out too.
__device__ __forceinline__ void quad_sync(int sub) { asm volatile("bar.sync %0, 128;" ::"r"(1 + sub) : "memory"); }

// Scales of this thread's four features in the fragments of features m0 ..: m0 + t / 4 + 8 i.
template <bool I8>
__device__ __forceinline__ void channel_scales(const RaggedParams &p, int e, int m0, float (&ch)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ((threadIdx.x & 31) >> 2) + 8 * i;
        ch[i] = (I8 && m < p.M) ? p.channel_scale[static_cast<int64_t>(e) * p.M + m] : 1.0f;
    }
}
// Scales of the item's rows, 32 i + lane, asked for before its sums are waited for: they would cost every chunk
// a trip to memory (48222 rows, 128 x 2112, INT8: 193 us so, 151 ahead of the wait).
template <bool I8, int CHUNKS>
__device__ __forceinline__ void row_scales(const RaggedParams &p, const RaggedItem &it, float (&rs)[CHUNKS]) {
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
        const int row = 32 * i + (threadIdx.x & 31);
        rs[i] = (I8 && row < it.n_valid) ? p.row_scale[it.row0 + row] : 1.0f;
    }
}
// A chunk of 16 rows: the 16 words of its two fragment loads to 8 words of packed pairs, for the two halves of 8
// rows four fragments (8 features each) each.  rs: the scales of its 32 rows (row_scales), of which it is the
// half `sub`.
template <bool I8, int TYPE>
__device__ __forceinline__ void pack_chunk(int sub, float rs, const float (&ch)[4], const uint32_t (&r)[16],
                                           uint32_t (&pk)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = 16 * sub + 8 * j + 2 * (threadIdx.x & 3);
        const float s0 = I8 ? __shfl_sync(0xffffffffu, rs, row) : 1.0f;
        const float s1 = I8 ? __shfl_sync(0xffffffffu, rs, row + 1) : 1.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = 8 * (i >> 1) + 4 * j + 2 * (i & 1);
            pk[4 * j + i] = pack2<TYPE>(ragged_value<I8>(r[at], ch[i], s0), ragged_value<I8>(r[at + 1], ch[i], s1));
        }
    }
}
// Stores a packed chunk of 16 rows from row c on.  q: this warp's 32 of the 128 features from mt0 on (M is a
// multiple of 8); stage: its four warps' two buffers, between which `flip` alternates, so that one barrier per
// chunk orders a buffer's writes after the reads of two chunks ago.  live: false after a wait has timed out.  TIGHT:
// a row's 16 bytes at a time, where two tiles' packed sums leave few registers (NA = 2: 4 bytes spilled, 120 with both
// rows together; the time is the same: 64 groups of ~256 rows, input gradients, 421 and 444 us against 433 and 435;
// 256 of ~128, 1178 against 1157); both rows together where the stores are the bound (NA = 1, 45231 rows, 224 x 4328:
// 5 to 15% less).
template <bool TIGHT>
__device__ __forceinline__ void store_chunk(const RaggedParams &p, const RaggedItem &it, int c, int mt0, int q, int sub,
                                            uint32_t stage, int flip, bool live, const uint32_t (&pk)[8]) {
    const int lane = threadIdx.x & 31;
    const uint32_t buf = stage + (flip & 1) * kStage16;
    {
        const int row = lane & 7, piece = 4 * q + (lane >> 3);  // row of a half, 16-byte piece of the row
        const uint32_t at = buf + row * 256 + ((piece ^ row) << 4);
        stmatrix_trans(at, {pk[0], pk[1], pk[2], pk[3]});
        stmatrix_trans(at + 8 * 256, {pk[4], pk[5], pk[6], pk[7]});
    }
    quad_sync(sub);
    // rows 4 q and 4 q + 1, then the next two
    const int piece = lane & 15;
    if constexpr (TIGHT) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = 4 * q + 2 * i + (lane >> 4), m = mt0 + 8 * piece;
            const uint4 v = lds128(buf + row * 256 + ((piece ^ (row & 7)) << 4));
            if (live && c + row < it.n_valid && m < p.M)
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.out) + (it.row0 + c + row) * p.ldo + m) = v;
        }
    } else {
        const int row = 4 * q + (lane >> 4);
        const uint32_t at = buf + row * 256;
        const uint4 lo = lds128(at + ((piece ^ (row & 7)) << 4));
        const uint4 hi = lds128(at + 512 + ((piece ^ ((row + 2) & 7)) << 4));
        if (live && mt0 + 8 * piece < p.M) {
            uint16_t *o = reinterpret_cast<uint16_t *>(p.out) + (it.row0 + c + row) * p.ldo + mt0 + 8 * piece;
            if (c + row < it.n_valid) *reinterpret_cast<uint4 *>(o) = lo;
            if (c + row + 2 < it.n_valid) *reinterpret_cast<uint4 *>(o + 2 * p.ldo) = hi;
        }
    }
}

// ---- forward / dgrad on CTA pairs ------------------------------------------------------------------
// The pair engine of gemm_2sm.cuh for one product.  A pair computes NA x 256 features x up to 256 rows; CTA r
// stages features 128 r.. of each 256 and half of the rows.
//   NA = 1: 6 stages of 16 KB + 16 KB, two TMEM slots of 256 columns, so that a segment's or an item's
//     epilogue always overlaps the next one's products.  INT8 sums are one segment: packed to 16 bits as they are
//     loaded (48222 rows, 128 x 2112: 151 us held as 32-bit words first, 107 so), or stored chunk by chunk (fp32).
//   NA = 2, 16-bit operands and results: 4 stages of 2 x 16 KB + 16 KB.  The staged bytes per product fall by a
//     quarter, for products that are bound by what L2 delivers to the SMs (ragged_plan).  Its one item fills TMEM,
//     so the epilogue packs the accumulators to 16 bits in registers, hands TMEM back and then stores.  INT8, whose
//     k-steps hold twice the products, has no such kernel: 8192 rows, 5120 x 5120, 131 us with NA = 1, 156 with 2;
//     8192 rows, 8192 x 8192, 340 and 346.
constexpr int kRpBN = 256;
// The rows of a k-step come in one box, of the height among eight (16, 32 .. 128 rows) that holds a CTA's half of
// the item's rows best: several small boxes cost more than their bytes (256 groups of 128 +- 11 rows, 5120 x
// 2560, NA = 1: 1.42 ms in boxes of 32 rows, 1.48 with a remainder of 8-row boxes, 1.32 so).
constexpr int kRpBoxStep = 16, kRpBoxes = 8;
struct RowMaps {
    CUtensorMap m[kRpBoxes];
};
template <int NA>
struct RpairCfg {
    static constexpr int kStages = NA == 1 ? 6 : 4;
    static constexpr int kStage = (NA + 1) * kRgOperand;
    static constexpr int kSlots = NA == 1 ? 2 : 1;
    static constexpr int kOutOff = kStages * kStage;  // staged 16-bit results
    static constexpr int kBarOff = kOutOff + kStage16All;
    static constexpr int kTileOff = kBarOff + 256;
    static constexpr int kSmem = 1024 + kTileOff + 4 * (kPmMaxE + 1) + 64;
    static_assert(8 * (2 * kStages + 2 * kSlots + 1) + 4 <= 256, "barrier area");
    static_assert(kSmem + 128 <= 232448, "shared memory per CTA (dynamic + the 128 static bytes)");
};

// Loads (first) or adds to acc the accumulator columns of this warp's share: chunks of 16 at 16 sub + stride i,
// those below n_valid; one lane per thread, or (FRAG) as fragments.
template <bool FRAG>
__device__ __forceinline__ void load_chunk(uint32_t t, uint32_t (&r)[16]) {
    if constexpr (FRAG) {
        tmem_ld_frag(t, r);
        tmem_ld_frag(t + (16u << 16), r + 8);
    } else {
        tmem_ld16(t, r);
    }
}
template <bool I8, bool FRAG, int CHUNKS>
__device__ __forceinline__ void add_segment(uint32_t t, int sub, int stride, int n_valid, bool first,
                                            uint32_t (&acc)[CHUNKS][16]) {
    if (first) {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
            if (16 * sub + stride * i < n_valid) load_chunk<FRAG>(t + 16 * sub + stride * i, acc[i]);  // warp-uniform
        tmem_ld_wait();
    } else {
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
            if (16 * sub + stride * i < n_valid) {
                uint32_t r[16];
                load_chunk<FRAG>(t + 16 * sub + stride * i, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    acc[i][j] = I8 ? acc[i][j] + r[j]
                                   : __float_as_uint(__uint_as_float(acc[i][j]) + __uint_as_float(r[j]));
            }
    }
}

// The warp's chunks (16 sub + 32 i) of its 32 features (mt0 + 32 q ..) from registers.
template <bool I8, int TYPE, int CHUNKS>
__device__ __forceinline__ void store_item(const RaggedParams &p, const RaggedItem &it, int sub, int q, int mt0,
                                           uint32_t stage, bool live, const float (&rs)[CHUNKS],
                                           const uint32_t (&acc)[CHUNKS][16]) {
    if constexpr (TYPE == BEAM_MOE_F32) {
        const int m = mt0 + 32 * q + (threadIdx.x & 31);
        const float channel = (I8 && m < p.M) ? p.channel_scale[static_cast<int64_t>(it.e) * p.M + m] : 1.0f;
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = 16 * sub + 32 * i;
            if (c < it.n_valid) {  // warp-uniform
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = ragged_value<I8>(acc[i][j], channel,
                                            I8 ? __shfl_sync(0xffffffffu, rs[i], 16 * sub + j) : 1.0f);
                if (live) store_cols(p, it, c, m, v);
            }
        }
    } else {
        float ch[4];
        channel_scales<I8>(p, it.e, mt0 + 32 * q, ch);
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
            const int c = 16 * sub + 32 * i;
            if (c < it.n_valid) {  // the same for the four warps
                uint32_t pk[8];
                pack_chunk<I8, TYPE>(sub, rs[i], ch, acc[i], pk);
                store_chunk<false>(p, it, c, mt0, q, sub, stage, i, live, pk);
            }
        }
        quad_sync(sub);  // the next item starts with the first buffer again
    }
}

// Items of one segment (NA = 2; INT8): this thread's 8 chunks of each of the item's NA accumulators, packed to 16
// bits (pack_chunk).
template <bool I8, int TYPE, int NA>
__device__ __forceinline__ void pack_item(const RaggedItem &it, uint32_t t, int sub, const float (&rs)[kRpBN / 32],
                                          const float (&ch)[NA][4], uint32_t (&pk)[NA][kRpBN / 32][8]) {
#pragma unroll
    for (int a = 0; a < NA; ++a) {
#pragma unroll
        for (int i = 0; i < kRpBN / 32; ++i) {
            const int c = 16 * sub + 32 * i;
            if (c < it.n_valid) {  // warp-uniform
                uint32_t r[16];
                load_chunk<true>(t + a * 256 + c, r);
                tmem_ld_wait();
                pack_chunk<I8, TYPE>(sub, rs[i], ch[a], r, pk[a][i]);
            }
        }
    }
}
// INT8's fp32 results: each chunk is stored as it is loaded.
__device__ __forceinline__ void store_i8_f32(const RaggedParams &p, const RaggedItem &it, uint32_t t, int sub, int m0,
                                             bool live, const float (&rs)[kRpBN / 32]) {
    const int m = m0 + (threadIdx.x & 31);
    const float channel = m < p.M ? p.channel_scale[static_cast<int64_t>(it.e) * p.M + m] : 1.0f;
#pragma unroll
    for (int i = 0; i < kRpBN / 32; ++i) {
        const int c = 16 * sub + 32 * i;
        if (c < it.n_valid) {  // warp-uniform
            uint32_t r[16];
            tmem_ld16(t + c, r);
            tmem_ld_wait();
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = ragged_value<true>(r[j], channel, __shfl_sync(0xffffffffu, rs[i], 16 * sub + j));
            if (live) store_cols(p, it, c, m, v);
        }
    }
}
template <int NA>
__device__ __forceinline__ void store_packed(const RaggedParams &p, const RaggedItem &it, int sub, int q, int mt0,
                                             uint32_t stage, bool live, const uint32_t (&pk)[NA][kRpBN / 32][8]) {
#pragma unroll
    for (int a = 0; a < NA; ++a) {
#pragma unroll
        for (int i = 0; i < kRpBN / 32; ++i)
            if (16 * sub + 32 * i < it.n_valid)  // the same for the four warps
                store_chunk<NA == 2>(p, it, 16 * sub + 32 * i, mt0 + a * kPairRows, q, sub, stage, i, live, pk[a][i]);
        quad_sync(sub);  // the buffers' turns start over
    }
}

template <bool I8, bool A_MN, int NA>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kRgThreads, 1)
    ragged_pair_kernel(const __grid_constant__ CUtensorMap tm_w,  // weights [E][N][K]
                       const __grid_constant__ RowMaps tm_b,      // rows [R][contraction], by box height
                       const RaggedParams p) {
    static_assert(NA == 1 || !I8, "INT8 runs with NA = 1");
    using C = RpairCfg<NA>;
    constexpr int kRound = I8 ? 32 : 16;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t gemm_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(gemm_smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *empty = full + kStages;
    uint64_t *acc_full = empty + kStages;
    uint64_t *acc_empty = acc_full + C::kSlots;
    uint64_t *drain = acc_empty + C::kSlots;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    int *tile_start = reinterpret_cast<int *>(smem + C::kTileOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = static_cast<int>(cluster_id_x()), n_pairs = static_cast<int>(cluster_count_x());
    const int n_mt = (p.M + NA * kPairRows - 1) / (NA * kPairRows);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < C::kSlots; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 2 * kGemmEpiWarps);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tensormap(&tm_w);
    }
    wait_for_stream();
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    ragged_prefix<kRpBN, false>(p, n_mt, false, tile_start);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total = tile_start[p.E], first = find_group(pair, tile_start, p.E);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer: this CTA's features and half of the rows
            const uint64_t pol_once = policy_evict_first(), pol_again = policy_evict_normal();
            const uint64_t pol_x = policy_evict_last();  // re-read by the other feature tiles
            const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
            constexpr int kElems = I8 ? 128 : 64;  // contraction elements per k-step
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            for (int item = pair, e = first; item < total && ok; item += n_pairs) {
                const RaggedItem it = ragged_item<kRpBN, kRound>(item, e, n_mt, tile_start, p);
                const uint64_t pol_w = it.once ? pol_once : pol_again;
                const int half = it.n_mma / 2;
                const int box = (half + kRpBoxStep - 1) / kRpBoxStep;  // 1..8
                const CUtensorMap *map_b = &tm_b.m[box - 1];
                const int b_row = static_cast<int>(it.row0) + static_cast<int>(rank) * half;
                const int a_row = it.mt * NA * kPairRows + static_cast<int>(rank) * kBM;
                const uint32_t pair_bytes =
                    2u * static_cast<uint32_t>(NA * kRgOperand + box * kRpBoxStep * kRgRowBytes);
                for (int kb = 0; kb < p.n_kb; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, p.timeout)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + stage * C::kStage;
                    const uint32_t bar = full_lead + 8u * static_cast<uint32_t>(stage);
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], pair_bytes);
#pragma unroll
                    for (int a = 0; a < NA; ++a) {
                        uint8_t *dst = sa + a * kRgOperand;
                        const int row = a_row + a * kPairRows;
                        if (A_MN) {
                            tma_load_3d_pair(dst, &tm_w, bar, row, kb * kElems, it.e, pol_w);
                            tma_load_3d_pair(dst + kRgOperand / 2, &tm_w, bar, row + 64, kb * kElems, it.e, pol_w);
                        } else {
                            tma_load_3d_pair(dst, &tm_w, bar, kb * kElems, row, it.e, pol_w);
                        }
                    }
                    tma_load_2d_pair(sa + NA * kRgOperand, map_b, bar, kb * kElems, b_row, pol_x);
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every stage this CTA loaded has been consumed by the pair's MMAs (so its bytes landed)
            for (int s = 0; s < kStages; ++s)
                if ((issued >> s) & 1u) mbar_wait(&empty[s], (issued_phase >> s) & 1u, p.timeout);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------- MMA issuer for the pair (leader CTA)
            int stage = 0;
            uint32_t phase = 0, uses = 0;
            bool ok = true;
            for (int item = pair, e = first; item < total && ok; item += n_pairs) {
                const RaggedItem it = ragged_item<kRpBN, kRound>(item, e, n_mt, tile_start, p);
                const uint32_t idesc = idesc_with_n(p.idesc, it.n_mma);
                for (int kb = 0; kb < p.n_kb && ok;) {
                    const int seg_end = NA == 1 ? min(p.n_kb, kb + p.seg_kb) : p.n_kb;
                    const uint32_t slot = uses % C::kSlots;
                    if (!mbar_wait(&acc_empty[slot], ((uses / C::kSlots) & 1u) ^ 1u, p.timeout)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + slot * 256;
                    for (bool start = true; kb < seg_end; ++kb, start = false) {
                        if (!mbar_wait(&full[stage], phase, p.timeout)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + stage * C::kStage);
                        const uint64_t db = umma_desc_sw128(sa + NA * kRgOperand);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of the contraction per instruction
                            const uint32_t accum = (!start || kk > 0) ? 1u : 0u;
#pragma unroll
                            for (int a = 0; a < NA; ++a) {
                                const uint32_t at = sa + a * kRgOperand;
                                const uint64_t da = A_MN ? umma_desc_mn_sw128(at) : umma_desc_sw128(at);
                                if (I8) umma_i8_pair(d + a * 256, da + 2 * kk, db + 2 * kk, idesc, accum);
                                else umma_bf16_pair(d + a * 256, da + (A_MN ? 128 : 2) * kk, db + 2 * kk, idesc, accum);
                            }
                        }
                        umma_commit_pair_both(&empty[stage]);
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    umma_commit_pair_both(&acc_full[slot]);
                    ++uses;
                }
            }
            umma_commit_pair_self(drain);
            mbar_wait(drain, 0, p.timeout);
        }
    } else {
        // ---------------- epilogue: two warps per lane quadrant, chunks of 16 rows at 16 sub + 32 i
        const int q = warp & 3, sub = (warp - 2) / 4;
        const uint32_t acc_empty_lead = mapa_shared(smem_u32(acc_empty), 0);
        const uint32_t t0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t stage_out = smem_u32(smem + C::kOutOff) + 2 * sub * kStage16;
        uint32_t uses = 0;
        bool ok = true;  // (the four warps of a quad stay together after a wait has timed out)
        for (int item = pair, e = first; item < total; item += n_pairs) {
            const RaggedItem it = ragged_item<kRpBN, kRound>(item, e, n_mt, tile_start, p);
            const int mt0 = it.mt * NA * kPairRows + static_cast<int>(rank) * kBM;  // this CTA's 128 features
            float rs[kRpBN / 32];
            row_scales<I8>(p, it, rs);
            if constexpr (NA == 1 && !I8) {
                uint32_t acc[kRpBN / 32][16];
                for (int kb = 0; kb < p.n_kb; kb += p.seg_kb, ++uses) {
                    ok = ok && mbar_wait(&acc_full[uses & 1], (uses >> 1) & 1u, p.timeout);
                    tc_fence_after();
                    const uint32_t t = t0 + (uses & 1) * 256;
                    if (p.out_type == BEAM_MOE_F32)
                        add_segment<I8, false, kRpBN / 32>(t, sub, 32, it.n_valid, kb == 0, acc);
                    else
                        add_segment<I8, true, kRpBN / 32>(t, sub, 32, it.n_valid, kb == 0, acc);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_async(acc_empty_lead + 8u * (uses & 1));
                }
                if (p.out_type == BEAM_MOE_BF16)
                    store_item<I8, BEAM_MOE_BF16, kRpBN / 32>(p, it, sub, q, mt0, stage_out, ok, rs, acc);
                else if (p.out_type == BEAM_MOE_F16)
                    store_item<I8, BEAM_MOE_F16, kRpBN / 32>(p, it, sub, q, mt0, stage_out, ok, rs, acc);
                else
                    store_item<I8, BEAM_MOE_F32, kRpBN / 32>(p, it, sub, q, mt0, stage_out, ok, rs, acc);
            } else {
                uint32_t pk[NA][kRpBN / 32][8];
                float ch[NA][4];
#pragma unroll
                for (int a = 0; a < NA; ++a) channel_scales<I8>(p, it.e, mt0 + 32 * q + a * kPairRows, ch[a]);
                const uint32_t slot = uses % C::kSlots, t = t0 + slot * 256;
                ok = ok && mbar_wait(&acc_full[slot], (uses / C::kSlots) & 1u, p.timeout);
                tc_fence_after();
                if (I8 && p.out_type == BEAM_MOE_F32) {
                    store_i8_f32(p, it, t, sub, mt0 + 32 * q, ok, rs);
                } else if (p.out_type == BEAM_MOE_BF16) {
                    pack_item<I8, BEAM_MOE_BF16, NA>(it, t, sub, rs, ch, pk);
                } else {
                    pack_item<I8, BEAM_MOE_F16, NA>(it, t, sub, rs, ch, pk);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_async(acc_empty_lead + 8u * slot);
                ++uses;
                if (!I8 || p.out_type != BEAM_MOE_F32) store_packed<NA>(p, it, sub, q, mt0, stage_out, ok, pk);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// ---- forward / dgrad with the contraction split over a cluster -------------------------------------
// For few rows per group, or few items: one product tile of 128 features x up to BN rows per cluster of
// S = 1, 2, 4 or 8 CTAs; CTA r takes k-steps [r n_kb / S, (r + 1) n_kb / S) and pushes 128 / S features of
// its partial sums to each CTA of the cluster over distributed shared memory; each CTA adds the S partial
// sums of its features in rank order (so results do not depend on timing) and stores them.
template <int BN, int STAGES>
struct RsplitCfg {
    static constexpr int kBox = BN == 32 ? 16 : 64;  // rows per B box (a box costs its producer as much as its bytes)
    static constexpr int kStage = kRgOperand + BN * kRgRowBytes;
    static constexpr int kRedOff = STAGES * kStage;           // the partial sums, fp32 (INT8: int32): partial_at
    static constexpr int kBarOff = kRedOff + BN * kBM * 4;
    static constexpr int kTileOff = kBarOff + 256;
    static constexpr int kSmem = 1024 + kTileOff + 4 * (kPmMaxE + 1) + 64;
    static constexpr int kSlot = BN < 32 ? 32 : BN;
    static_assert(8 * (2 * STAGES + 4 + 2 + 1) + 4 <= 256, "barrier area");
    static_assert(kStage % 1024 == 0 && kSmem + 128 <= 232448, "shared memory per CTA");
    static_assert(kStage16All <= BN * kBM * 4, "staged 16-bit results lie in the partial sums' place");
};
// 16 bytes to shared memory of a CTA of the cluster; they complete on an mbarrier of that CTA, so neither side
// needs a fence (plain remote stores with a cluster-scope release took about 3 us per item).
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                            uint32_t bar) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.u32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
        "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Partial sums in a CTA's shared memory: [S][F = 128 / S features][BN rows], four rows (16 bytes) at a time,
// those of feature f at place (rows / 4) ^ (f & 7), so that neighbouring features fall into different banks.
template <int BN>
__device__ __forceinline__ uint32_t partial_at(uint32_t feature, uint32_t quad) {
    return feature * (BN * 4) + ((quad ^ (feature & 7u)) << 4);
}

// This CTA's features (m0 ..) of one item: the S partial sums of four rows of a feature per thread and step, added
// in rank order; 16-bit results are paired with the neighbouring lane's feature.
template <bool I8, int BN, int TYPE>
__device__ __forceinline__ void reduce_store(const RaggedParams &p, const RaggedItem &it, uint32_t buf, int S, int F,
                                             int m0, int tid) {
    const int log_f = 31 - __clz(F);
    const int total = ((it.n_valid + 3) >> 2) << log_f;  // four-row pieces
    const int f = tid & (F - 1), m = m0 + f;             // F divides 256: a thread keeps its feature
    const float channel = (I8 && m < p.M) ? p.channel_scale[static_cast<int64_t>(it.e) * p.M + m] : 1.0f;
    for (int idx = tid; idx - (tid & 31) < total; idx += 32 * kGemmEpiWarps) {  // warp-uniform
        const int quad = idx >> log_f;
        const bool live = idx < total && m < p.M;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (live) {
            uint4 sum = lds128(buf + partial_at<BN>(f, quad));
            for (int s = 1; s < S; ++s) {
                const uint4 u = lds128(buf + partial_at<BN>(s * F + f, quad));
                if constexpr (I8) {
                    sum = make_uint4(sum.x + u.x, sum.y + u.y, sum.z + u.z, sum.w + u.w);
                } else {
                    sum = make_uint4(__float_as_uint(__uint_as_float(sum.x) + __uint_as_float(u.x)),
                                     __float_as_uint(__uint_as_float(sum.y) + __uint_as_float(u.y)),
                                     __float_as_uint(__uint_as_float(sum.z) + __uint_as_float(u.z)),
                                     __float_as_uint(__uint_as_float(sum.w) + __uint_as_float(u.w)));
                }
            }
            const uint32_t w[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * quad + j;
                const float row = (I8 && c < it.n_valid) ? p.row_scale[it.row0 + c] : 1.0f;
                v[j] = ragged_value<I8>(w[j], channel, row);
            }
        }
        const int left = live ? it.n_valid - 4 * quad : 0;
        if constexpr (TYPE == BEAM_MOE_F32) {
            float *o = reinterpret_cast<float *>(p.out) + (it.row0 + 4 * quad) * p.ldo + m;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left) o[j * p.ldo] = v[j];
        } else {
            const int odd = tid & 1;
            uint16_t *o = reinterpret_cast<uint16_t *>(p.out) + (it.row0 + 4 * quad + odd) * p.ldo + (m & ~1);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                const uint32_t pr = odd ? pack2<TYPE>(got, v[j + 1]) : pack2<TYPE>(v[j], got);
                if (j + odd < left) *reinterpret_cast<uint32_t *>(o + j * p.ldo) = pr;
            }
        }
    }
}

template <bool I8, bool A_MN, int BN, int STAGES>
__global__ void __launch_bounds__(kRgThreads, 1)
    ragged_split_kernel(const __grid_constant__ CUtensorMap tm_w,  // weights [E][N][K]
                        const __grid_constant__ CUtensorMap tm_b,  // rows [R][contraction], kBox-row box
                        const RaggedParams p) {
    using C = RsplitCfg<BN, STAGES>;
    constexpr int kChunks = (BN + 31) / 32;
    extern __shared__ uint8_t gemm_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(gemm_smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *red_full = acc_empty + 2;   // all S partial sums of this CTA's features have arrived
    uint64_t *red_empty = red_full + 1;   // every CTA of the cluster has read its partial sums
    uint64_t *drain = red_empty + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    int *tile_start = reinterpret_cast<int *>(smem + C::kTileOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t S;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
    const uint32_t rank = cluster_ctarank();
    const int cluster = static_cast<int>(cluster_id_x()), n_clusters = static_cast<int>(cluster_count_x());
    const int n_mt = (p.M + kBM - 1) / kBM;
    const int kb0 = static_cast<int>(rank) * p.n_kb / static_cast<int>(S);
    const int kb1 = (static_cast<int>(rank) + 1) * p.n_kb / static_cast<int>(S);  // S <= n_kb: never empty

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], kGemmEpiWarps);
        }
        mbar_init(red_full, 1);
        mbar_init(red_empty, kGemmEpiWarps * S);
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_b);
    }
    wait_for_stream();
    if (warp == 1) {
        tmem_alloc(tmem_slot, 2 * C::kSlot);
        tmem_relinquish();
    }
    ragged_prefix<BN, false>(p, n_mt, false, tile_start);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();  // the epilogue waits for the other CTAs' barriers before it signals them; nobody else does
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total = tile_start[p.E], first = find_group(cluster, tile_start, p.E);

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol_once = policy_evict_first(), pol_again = policy_evict_normal();
            const uint64_t pol_x = policy_evict_last();  // re-read by the other feature tiles
            constexpr int kElems = I8 ? 128 : 64;
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            for (int item = cluster, e = first; item < total && ok; item += n_clusters) {
                const RaggedItem it = ragged_item<BN, 16>(item, e, n_mt, tile_start, p);
                const uint64_t pol_w = it.once ? pol_once : pol_again;
                const int nbox = (it.n_mma + C::kBox - 1) / C::kBox;
                const int a_row = it.mt * kBM;
                const uint32_t bytes = static_cast<uint32_t>(kRgOperand + nbox * C::kBox * kRgRowBytes);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, p.timeout)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + stage * C::kStage;
                    mbar_arrive_expect_tx(&full[stage], bytes);
                    if (A_MN) {
                        tma_load_3d(sa, &tm_w, &full[stage], a_row, kb * kElems, it.e, pol_w);
                        tma_load_3d(sa + kRgOperand / 2, &tm_w, &full[stage], a_row + 64, kb * kElems, it.e, pol_w);
                    } else {
                        tma_load_3d(sa, &tm_w, &full[stage], kb * kElems, a_row, it.e, pol_w);
                    }
                    for (int b = 0; b < nbox; ++b)
                        tma_load_2d(sa + kRgOperand + b * C::kBox * kRgRowBytes, &tm_b, &full[stage], kb * kElems,
                                    static_cast<int>(it.row0) + b * C::kBox, pol_x);
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < STAGES; ++s)
                if ((issued >> s) & 1u) mbar_wait(&empty[s], (issued_phase >> s) & 1u, p.timeout);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, uses = 0;
            bool ok = true;
            for (int item = cluster, e = first; item < total && ok; item += n_clusters) {
                const RaggedItem it = ragged_item<BN, 16>(item, e, n_mt, tile_start, p);
                const uint32_t idesc = idesc_with_n(p.idesc, it.n_mma);
                for (int kb = kb0; kb < kb1 && ok;) {
                    const int seg_end = min(kb1, kb + p.seg_kb);
                    if (!mbar_wait(&acc_empty[uses & 1], ((uses >> 1) & 1u) ^ 1u, p.timeout)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + (uses & 1) * C::kSlot;
                    for (bool start = true; kb < seg_end; ++kb, start = false) {
                        if (!mbar_wait(&full[stage], phase, p.timeout)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + stage * C::kStage);
                        const uint64_t da = A_MN ? umma_desc_mn_sw128(sa) : umma_desc_sw128(sa);
                        const uint64_t db = umma_desc_sw128(sa + kRgOperand);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t accum = (!start || kk > 0) ? 1u : 0u;
                            if (I8) umma_i8(d, da + 2 * kk, db + 2 * kk, idesc, accum);
                            else umma_bf16(d, da + (A_MN ? 128 : 2) * kk, db + 2 * kk, idesc, accum);
                        }
                        umma_commit(&empty[stage]);
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    umma_commit(&acc_full[uses & 1]);
                    ++uses;
                }
            }
            umma_commit(drain);
            mbar_wait(drain, 0, p.timeout);
        }
    } else {
        const int q = warp & 3, sub = (warp - 2) / 4;
        const int F = kBM / static_cast<int>(S);
        const uint32_t buf = smem_u32(smem + C::kRedOff);
        // this thread's feature q * 32 + lane belongs to CTA `dst`, which keeps it at index f of its F
        const uint32_t dst = static_cast<uint32_t>(q * 32 + lane) / F;
        const uint32_t f = rank * F + static_cast<uint32_t>(q * 32 + lane) % F;
        const uint32_t push = mapa_shared(buf, dst), push_bar = mapa_shared(smem_u32(red_full), dst);
        uint32_t uses = 0, n_item = 0;
        bool ok = true, joined = false;  // joined: the other CTAs' barriers are known to be initialised
        for (int item = cluster, e = first; item < total; item += n_clusters, ++n_item) {
            const RaggedItem it = ragged_item<BN, 16>(item, e, n_mt, tile_start, p);
            uint32_t acc[kChunks][16];
            float rs[kChunks];
            if (S == 1) row_scales<I8>(p, it, rs);
            for (int kb = kb0; kb < kb1; kb += p.seg_kb, ++uses) {
                ok = ok && mbar_wait(&acc_full[uses & 1], (uses >> 1) & 1u, p.timeout);
                tc_fence_after();
                const uint32_t t = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + (uses & 1) * C::kSlot;
                if (S == 1 && p.out_type != BEAM_MOE_F32)
                    add_segment<I8, true, kChunks>(t, sub, 32, it.n_valid, kb == kb0, acc);
                else
                    add_segment<I8, false, kChunks>(t, sub, 32, it.n_valid, kb == kb0, acc);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[uses & 1]);
            }
            if (S == 1) {  // (the four warps of a quad stay together after a wait has timed out)
                const uint32_t stage_out = buf + 2 * sub * kStage16;  // (no partial sums are exchanged)
                if (p.out_type == BEAM_MOE_BF16)
                    store_item<I8, BEAM_MOE_BF16, kChunks>(p, it, sub, q, it.mt * kBM, stage_out, ok, rs, acc);
                else if (p.out_type == BEAM_MOE_F16)
                    store_item<I8, BEAM_MOE_F16, kChunks>(p, it, sub, q, it.mt * kBM, stage_out, ok, rs, acc);
                else
                    store_item<I8, BEAM_MOE_F32, kChunks>(p, it, sub, q, it.mt * kBM, stage_out, ok, rs, acc);
                continue;
            }
            if (!ok) break;
            if (!joined) {
                cluster_wait();
                joined = true;
            }
            if (threadIdx.x == 64)  // what the S CTAs push here for this item
                mbar_arrive_expect_tx(red_full, static_cast<uint32_t>(kBM * ((it.n_valid + 3) >> 2) * 16));
            // the last item's partial sums have been read everywhere, then these are pushed
            ok = mbar_wait(red_empty, (n_item & 1u) ^ 1u, p.timeout);
            if (!ok) break;
            acquire_smem();
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int c = 16 * sub + 32 * i;
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    if (c + j < it.n_valid)
                        st_async_v4(push + partial_at<BN>(f, static_cast<uint32_t>(c + j) >> 2), acc[i][j],
                                    acc[i][j + 1], acc[i][j + 2], acc[i][j + 3], push_bar);
            }
            ok = mbar_wait(red_full, n_item & 1u, p.timeout);
            if (!ok) break;
            acquire_smem();
            const int tid = static_cast<int>(threadIdx.x) - 64;
            const int m0 = it.mt * kBM + static_cast<int>(rank) * F;
            if (p.out_type == BEAM_MOE_BF16) reduce_store<I8, BN, BEAM_MOE_BF16>(p, it, buf, S, F, m0, tid);
            else if (p.out_type == BEAM_MOE_F16) reduce_store<I8, BN, BEAM_MOE_F16>(p, it, buf, S, F, m0, tid);
            else reduce_store<I8, BN, BEAM_MOE_F32>(p, it, buf, S, F, m0, tid);
            __syncwarp();  // this warp has read its sums: one arrival per CTA of the cluster
            if (item + n_clusters < total && lane < static_cast<int>(S))
                mbar_release_smem(mapa_shared(smem_u32(red_empty), lane));
        }
        if (!joined) cluster_wait();
    }
    __syncwarp();
    if (warp < 2) cluster_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while another may still push to it or signal it
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, 2 * C::kSlot);
}

// ---- wgrad on CTA pairs ----------------------------------------------------------------------------
// dw[e][n][k] tiles of 256 x 256 NB: the contraction runs over the group's rows in k-steps of 64, dy^T is the
// MMA's A (CTA r: columns n 128 r..), x^T its B (CTA r: half of each 256 columns k), both MN-major.  The rows
// of a group's last k-step that belong to the next group must not enter the sums, and zero times a NaN there
// would: a helper warp clears them in shared memory.  A staged row is one 128-byte line of each box
// (swizzling permutes within the line), so rows v.. of a box are the contiguous bytes [128 v, ...), and
// only the rows up to the next multiple of 16 (one instruction's contraction) are cleared and multiplied.
//   full[s] (leader, two arrivals)  a whole k-step's loads of both CTAs complete on it directly, both
//            arrivals being the leader's producer's; for a k-step to clear the two helpers arrive on it
//   tail[s]  this CTA's loads of a k-step to clear have landed
// No producer arrives on the other CTA's barrier: one such release at cluster scope per k-step, which waits
// for the thread's earlier memory operations, held the ring at 700 TFLOP/s (with or without the products).  The helper
// of the peer does, with a release of shared memory alone.
//
// The epilogue stages 32 rows x 128 bytes per warp at a time, swizzled, and stores them with TMA, which clips
// at N and K and, for `accumulate`, adds (FP32).  Groups without rows store zeros.
//   NB = 1: 5 stages of 16 KB + 16 KB, two TMEM slots, two staging buffers per warp; sums longer than
//     seg_kb k-steps are cut into segments, added in registers.
//   NB = 2: 4 stages of 16 KB + 2 x 16 KB, so a quarter fewer bytes from L2, which bounds both long groups
//     (L2 to the SMs) and short ones (loads and stores together); one item fills TMEM and each warp has one
//     staging buffer.  fp32 results of more than seg_kb k-steps are flushed by TMA adds.
// With `splits` > 1 split s takes its share of each group's k-steps and stores FP32 partial sums at group
// index s E + e of a [splits E][N][K] workspace, which ragged_join_kernel adds in order.
constexpr int kRwThreads = 384;    // warp 0 TMA, warp 1 MMA, warp 2 helper, warp 3 idle, warps 4..11 epilogue
constexpr int kRwStageOut = 4096;  // one staged output chunk: 32 rows of 128 bytes
template <int NB>
struct RwgradCfg {
    static constexpr int kStages = NB == 1 ? 5 : 4;
    static constexpr int kStage = (1 + NB) * kRgOperand;
    static constexpr int kSlots = NB == 1 ? 2 : 1;
    static constexpr int kOutBufs = NB == 1 ? 2 : 1;  // per warp
    static constexpr int kOutOff = kStages * kStage;
    static constexpr int kBarOff = kOutOff + kGemmEpiWarps * kOutBufs * kRwStageOut;
    static constexpr int kTileOff = kBarOff + 256;
    static constexpr int kSmem = 1024 + kTileOff + 4 * (kPmMaxE + 1) + 64;
    static_assert(8 * (3 * kStages + 2 * kSlots + 1) + 4 <= 256, "barrier area");
    static_assert(kSmem + 128 <= 232448, "shared memory per CTA (dynamic + the 128 static bytes)");
};

struct WgradItem {
    int e, n0, k0;
    int group;             // group index of the stored tile: split * E + e
    int64_t row0;
    int rows;              // rows of this item's share of the group (its first row is row0)
};
struct WgradParams {
    RaggedParams g;  // M = N of the product; n_kb unused
    int K, n_mt, n_nt, splits;
    uint32_t nt_inv;  // ceil(2^32 / n_nt): local / n_nt = local * nt_inv >> 32, exact for local * n_nt < 2^32
    int accumulate;  // FP32 output: add to it, groups without rows are left alone
    int dy_blocks, x_blocks;  // the operand's map has 64-column blocks: 128 columns in one load
};

// Every role decodes every item, and a short group's item is over in ~2000 cycles: no search from the start and
// no slow division here (with both, 64 groups of 32 rows took 250 us without their stores instead of 135).
template <int NB>
__device__ __forceinline__ WgradItem wgrad_item(int item, int &e, const int *tile_start, const WgradParams &p) {
    WgradItem it;
    while (tile_start[e + 1] <= item) ++e;
    it.e = e;
    uint32_t local = static_cast<uint32_t>(item - tile_start[e]);
    const int rows = group_rows(p.g, e);
    it.row0 = group_begin(p.g, e);
    it.rows = rows;
    it.group = e;
    if (p.splits > 1) {
        const uint32_t tiles = static_cast<uint32_t>(p.n_mt * p.n_nt), split = local / tiles;
        const uint32_t steps = static_cast<uint32_t>((rows + 63) / 64), n = static_cast<uint32_t>(p.splits);
        local -= split * tiles;
        const int r0 = static_cast<int>(steps * split / n) * 64;  // steps <= 2^18, splits <= 64
        const int r1 = min(rows, static_cast<int>(steps * (split + 1) / n) * 64);
        it.row0 += r0;
        it.rows = max(0, r1 - r0);
        it.group = static_cast<int>(split) * p.g.E + e;
    }
    const uint32_t mt = p.n_nt == 1 ? local : __umulhi(local, p.nt_inv);
    it.n0 = static_cast<int>(mt) * kPairRows;
    it.k0 = static_cast<int>(local - mt * static_cast<uint32_t>(p.n_nt)) * (256 * NB);
    return it;
}
// Columns of the product at column k0 of K (256, or 128 where no more are left; 0: none).
__device__ __forceinline__ int wgrad_cols(int k0, int K) { return K - k0 > 128 ? 256 : (K > k0 ? 128 : 0); }

// A k-step of v rows of the group (64 or more: whole): whether its last instruction meets rows behind it.
__device__ __forceinline__ bool needs_clearing(int v) { return v < 64 && (v & 15); }

// (evict-first: results of a size that does not stay in L2 anyway, 6% off the fp32 case)
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int c0, int c1, int c2,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], %5;" ::"l"(map),
        "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap *map, const void *src, int c0, int c1, int c2) {
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
        "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
        : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// A warp's output: 128 bytes of each of its 32 rows (one per lane) at a time go through a staging buffer.
template <int BUFS>
struct WgradOut {
    const CUtensorMap *map;
    uint8_t *stage;
    uint64_t policy;
    uint32_t n_out;  // chunks so far

    // Columns k.. of rows n.. of group `group`; word(i): the i-th of this lane's 32 words.
    template <typename F>
    __device__ __forceinline__ void chunk(int k, int n, int group, bool add, F word) {
        const int lane = threadIdx.x & 31;
        uint8_t *src = stage + (BUFS == 1 ? 0 : (n_out & 1) * kRwStageOut);
        ++n_out;
        if (lane == 0) bulk_wait_read<BUFS - 1>();  // the store that last used this buffer has read it
        __syncwarp();
        const uint32_t buf = smem_u32(src) + lane * 128;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sts128(buf + ((j ^ (lane & 7)) << 4),
                   make_uint4(word(4 * j), word(4 * j + 1), word(4 * j + 2), word(4 * j + 3)));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (add) tma_add_3d(map, src, k, n, group);
            else tma_store_3d(map, src, k, n, group, policy);
            bulk_commit();
        }
    }
};

// 128 columns (those below k_end) of fp32 accumulators, in `TYPE`.
template <int TYPE, int BUFS>
__device__ __forceinline__ void wgrad_store(WgradOut<BUFS> &out, int group, int n, int k, int k_end, bool add,
                                            const uint32_t (&acc)[8][16]) {
    constexpr int kCols = TYPE == BEAM_MOE_F32 ? 32 : 64;  // columns per 128 bytes
#pragma unroll
    for (int b = 0; b < 128 / kCols; ++b) {
        if (k + b * kCols < k_end) {  // warp-uniform
            out.chunk(k + b * kCols, n, group, add, [&](int i) {
                if constexpr (TYPE == BEAM_MOE_F32) {
                    const int c = b * 32 + i;
                    return acc[c / 16][c % 16];
                } else {
                    const int c = b * 64 + 2 * i;
                    return pack2<TYPE>(__uint_as_float(acc[c / 16][c % 16]), __uint_as_float(acc[c / 16][c % 16 + 1]));
                }
            });
        }
    }
}

// NB = 2, 16-bit results: the two products' accumulators packed to 16 bits, TMEM handed back, then stored.
template <int TYPE>
__device__ __forceinline__ void wgrad_pack_store(WgradOut<1> &out, const WgradItem &it, int K, int sub, int n,
                                                 bool live, bool rows, uint32_t t0, uint32_t acc_empty_lead) {
    uint32_t pk[2][8][8];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int cols = wgrad_cols(it.k0 + 256 * b, K) / 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (rows && 16 * i < cols) {  // warp-uniform
                uint32_t r[16];
                tmem_ld16(t0 + 256 * b + cols * sub + 16 * i, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    pk[b][i][j] = pack2<TYPE>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) pk[b][i][j] = 0u;
            }
        }
    }
    if (rows) {
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive_async(acc_empty_lead);
    }
    if (!live) return;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int cols = wgrad_cols(it.k0 + 256 * b, K) / 2;
        const int k = it.k0 + 256 * b + cols * sub, k_end = min(K, k + cols);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (k + 64 * c < k_end)
                out.chunk(k + 64 * c, n, it.group, false, [&](int i) { return pk[b][c * 4 + i / 8][i % 8]; });
        }
    }
}

template <int NB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kRwThreads, 1)
    ragged_wgrad_kernel(const __grid_constant__ CUtensorMap tm_dy,  // [R][N], box 64 x 64
                        const __grid_constant__ CUtensorMap tm_x,   // [R][K], box 64 x 64
                        const __grid_constant__ CUtensorMap tm_dw,  // [groups][N][K], box 32 rows x 128 bytes
                        const WgradParams p) {
    using C = RwgradCfg<NB>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t gemm_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(gemm_smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *empty = full + kStages;
    uint64_t *acc_full = empty + kStages;
    uint64_t *acc_empty = acc_full + C::kSlots;
    uint64_t *tail = acc_empty + C::kSlots;
    uint64_t *drain = tail + kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    int *tile_start = reinterpret_cast<int *>(smem + C::kTileOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = static_cast<int>(cluster_id_x()), n_pairs = static_cast<int>(cluster_count_x());
    const long long timeout = p.g.timeout;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 1);
            mbar_init(&tail[s], 1);
        }
        for (int a = 0; a < C::kSlots; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 2 * kGemmEpiWarps);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        prefetch_tensormap(&tm_dy);
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_dw);
    }
    wait_for_stream();
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    ragged_prefix<256, true>(p.g, p.n_mt * p.n_nt * p.splits, p.accumulate != 0, tile_start);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total = tile_start[p.g.E], first = find_group(pair, tile_start, p.g.E);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer
            const uint64_t pol = policy_evict_normal();
            const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
            const uint32_t tail_own = mapa_shared(smem_u32(tail), rank);
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            for (int item = pair, e = first; item < total && ok; item += n_pairs) {
                const WgradItem it = wgrad_item<NB>(item, e, tile_start, p);
                const int a_col = it.n0 + static_cast<int>(rank) * kBM;
                int nbox[NB], b_col[NB];  // 64-column boxes of x per CTA
                int boxes = 2;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const int cols = wgrad_cols(it.k0 + 256 * j, p.K);
                    nbox[j] = p.x_blocks && cols ? 2 : cols / 128;  // (blocks: also those a half tile does not use)
                    b_col[j] = it.k0 + 256 * j + static_cast<int>(rank) * (cols / 2);
                    boxes += nbox[j];
                }
                const uint32_t bytes = static_cast<uint32_t>(boxes * (kRgOperand / 2));
                for (int r = 0; r < it.rows; r += 64) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, timeout)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + stage * C::kStage;
                    const int row = static_cast<int>(it.row0) + r;
                    uint32_t bar = full_lead + 8u * static_cast<uint32_t>(stage);
                    if (needs_clearing(it.rows - r)) {
                        bar = tail_own + 8u * static_cast<uint32_t>(stage);
                        mbar_arrive_expect_tx(&tail[stage], bytes);
                    } else if (rank == 0) {
                        mbar_arrive_expect_tx(&full[stage], 2u * bytes);
                        mbar_arrive(&full[stage]);
                    }
                    if (p.dy_blocks) {
                        tma_load_3d_pair(sa, &tm_dy, bar, 0, row, a_col / 64, pol);
                    } else {
                        tma_load_2d_pair(sa, &tm_dy, bar, a_col, row, pol);
                        tma_load_2d_pair(sa + kRgOperand / 2, &tm_dy, bar, a_col + 64, row, pol);
                    }
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        uint8_t *sb = sa + (1 + j) * kRgOperand;
                        if (p.x_blocks) {
                            if (nbox[j]) tma_load_3d_pair(sb, &tm_x, bar, 0, row, b_col[j] / 64, pol);
                        } else {
                            for (int b = 0; b < nbox[j]; ++b)
                                tma_load_2d_pair(sb + b * (kRgOperand / 2), &tm_x, bar, b_col[j] + 64 * b, row, pol);
                        }
                    }
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            for (int s = 0; s < kStages; ++s)
                if ((issued >> s) & 1u) mbar_wait(&empty[s], (issued_phase >> s) & 1u, timeout);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------- MMA issuer for the pair
            int stage = 0;
            uint32_t phase = 0, uses = 0;
            bool ok = true;
            for (int item = pair, e = first; item < total && ok; item += n_pairs) {
                const WgradItem it = wgrad_item<NB>(item, e, tile_start, p);
                uint32_t idesc[NB];
                int n_b = 0;  // products of the item
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const int cols = wgrad_cols(it.k0 + 256 * j, p.K);
                    idesc[j] = idesc_with_n(p.g.idesc, cols);
                    n_b += cols > 0;
                }
                const int n_kb = (it.rows + 63) / 64;
                for (int kb = 0; kb < n_kb && ok;) {
                    const int seg_end = min(n_kb, kb + p.g.seg_kb);
                    const uint32_t slot = uses % C::kSlots;
                    if (!mbar_wait(&acc_empty[slot], ((uses / C::kSlots) & 1u) ^ 1u, timeout)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + slot * 256;
                    for (bool start = true; kb < seg_end; ++kb, start = false) {
                        if (!mbar_wait(&full[stage], phase, timeout)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + stage * C::kStage);
                        if (needs_clearing(it.rows - kb * 64)) acquire_smem();
                        const uint64_t da = umma_desc_mn_sw128(sa);
                        const int n_mma16 = min(4, (it.rows - kb * 64 + 15) / 16);
                        for (int kk = 0; kk < n_mma16; ++kk)
#pragma unroll
                            for (int j = 0; j < NB; ++j)
                                if (j < n_b)
                                    umma_bf16_pair(d + 256 * j, da + 128 * kk,
                                                   umma_desc_mn_sw128(sa + (1 + j) * kRgOperand) + 128 * kk, idesc[j],
                                                   (!start || kk > 0) ? 1u : 0u);
                        umma_commit_pair_both(&empty[stage]);
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    umma_commit_pair_both(&acc_full[slot]);
                    ++uses;
                }
            }
            umma_commit_pair_self(drain);
            mbar_wait(drain, 0, timeout);
        }
    } else if (warp == 2) {
        // ---------------- helper: clears the rows behind the group in its last k-step
        const uint32_t full_lead = mapa_shared(smem_u32(full), 0);
        uint32_t steps = 0, phases = 0;  // k-steps up to this item's end; per stage, the phase of `tail`
        long long limit = timeout;       // one for each item that it lets pass, and one for its own
        for (int item = pair, e = first; item < total; item += n_pairs) {
            const WgradItem it = wgrad_item<NB>(item, e, tile_start, p);
            if (it.rows == 0) continue;
            const uint32_t n_kb = static_cast<uint32_t>((it.rows + 63) / 64);
            steps += n_kb;
            const int v = it.rows - static_cast<int>(n_kb - 1) * 64;
            if (!needs_clearing(v)) {
                limit += timeout;
                continue;
            }
            const uint32_t stage = (steps - 1) % kStages;
            const uint32_t phase = (phases >> stage) & 1u;
            phases ^= 1u << stage;
            if (!mbar_wait(&tail[stage], phase, limit)) break;
            limit = timeout;
            const uint32_t sa = smem_u32(smem + stage * C::kStage);
            const int lines = ((v + 15) & ~15) - v;  // 1..15 lines of 128 bytes per box
            // every box of the stage (those not loaded for this item hold nothing that is used)
            for (int i = lane; i < 2 * (1 + NB) * lines * 8; i += 32) {
                const int box = i / (lines * 8), at = i - box * lines * 8;
                sts128(sa + box * (kRgOperand / 2) + v * 128 + at * 16, make_uint4(0u, 0u, 0u, 0u));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) mbar_arrive(&full[stage]);
                else mbar_release_smem(full_lead + 8u * stage);
            }
        }
    } else if (warp >= 4) {
        // ---------------- epilogue: lanes = rows n, two warps per quadrant share a product's columns
        const int q = warp & 3, sub = (warp - 4) / 4;
        const uint32_t acc_empty_lead = mapa_shared(smem_u32(acc_empty), 0);
        const uint32_t t0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        WgradOut<C::kOutBufs> out{&tm_dw, smem + C::kOutOff + (warp - 4) * C::kOutBufs * kRwStageOut,
                                  policy_evict_first(), 0u};
        uint32_t uses = 0;
        bool ok = true;
        for (int item = pair, e = first; item < total && ok; item += n_pairs) {
            const WgradItem it = wgrad_item<NB>(item, e, tile_start, p);
            const int n_kb = (it.rows + 63) / 64;
            const int n = it.n0 + static_cast<int>(rank) * kBM + q * 32;
            const bool live = n < p.g.M;  // warp-uniform
            if constexpr (NB == 1) {
                const int cols = wgrad_cols(it.k0, p.K) / 2;  // this warp's columns: [cols sub, cols (sub + 1))
                uint32_t acc[8][16];
                if (n_kb == 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[i][j] = 0u;
                }
                for (int kb = 0; kb < n_kb; kb += p.g.seg_kb, ++uses) {
                    if (!mbar_wait(&acc_full[uses & 1], (uses >> 1) & 1u, timeout)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    add_segment<false, false, 8>(t0 + (uses & 1) * 256 + cols * sub, 0, 16, cols, kb == 0, acc);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_async(acc_empty_lead + 8u * (uses & 1));
                }
                if (!ok) break;
                const int k = it.k0 + cols * sub, k_end = min(p.K, k + cols);
                if (live) {
                    if (p.g.out_type == BEAM_MOE_BF16)
                        wgrad_store<BEAM_MOE_BF16>(out, it.group, n, k, k_end, false, acc);
                    else if (p.g.out_type == BEAM_MOE_F16)
                        wgrad_store<BEAM_MOE_F16>(out, it.group, n, k, k_end, false, acc);
                    else
                        wgrad_store<BEAM_MOE_F32>(out, it.group, n, k, k_end, p.accumulate != 0, acc);
                }
            } else if (p.g.out_type == BEAM_MOE_F32) {
                // one pass per segment (one without sums for a group without rows): store, or add
                for (int kb = 0; kb == 0 || kb < n_kb; kb += p.g.seg_kb) {
                    if (n_kb > 0) {
                        ok = mbar_wait(acc_full, uses & 1u, timeout);
                        if (!ok) break;
                        tc_fence_after();
                        if (kb > 0 && lane == 0) bulk_wait_all();  // this segment's adds follow the last one's stores
                        __syncwarp();
                    }
#pragma unroll 1
                    for (int b = 0; b < 2; ++b) {
                        const int cols = wgrad_cols(it.k0 + 256 * b, p.K) / 2;
                        const int k = it.k0 + 256 * b + cols * sub;
#pragma unroll 1
                        for (int c = 0; c < cols && k + c < p.K; c += 32) {
                            uint32_t r[2][16] = {};
                            if (n_kb > 0) {
                                tmem_ld16(t0 + 256 * b + cols * sub + c, r[0]);
                                tmem_ld16(t0 + 256 * b + cols * sub + c + 16, r[1]);
                                tmem_ld_wait();
                            }
                            if (live)
                                out.chunk(k + c, n, it.group, kb > 0 || p.accumulate != 0,
                                          [&](int i) { return r[i / 16][i % 16]; });
                        }
                    }
                    if (n_kb > 0) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_async(acc_empty_lead);
                        ++uses;
                    }
                }
            } else {
                if (n_kb > 0) {
                    ok = mbar_wait(acc_full, uses & 1u, timeout);
                    if (!ok) break;
                    tc_fence_after();
                    ++uses;
                }
                if (p.g.out_type == BEAM_MOE_BF16)
                    wgrad_pack_store<BEAM_MOE_BF16>(out, it, p.K, sub, n, live, n_kb > 0, t0, acc_empty_lead);
                else
                    wgrad_pack_store<BEAM_MOE_F16>(out, it, p.K, sub, n, live, n_kb > 0, t0, acc_empty_lead);
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// dw = (accumulate ? dw : 0) + the FP32 partial sums of `splits` splits in order, n values each.  Where it
// accumulates, groups without rows are left alone (a sum of zeros would turn -0 into 0); rows are only split where
// few weights are, so the index of four values fits 32 bits.
template <int TYPE>
__global__ void __launch_bounds__(256) ragged_join_kernel(const float4 *__restrict__ part, int splits, int64_t n4,
                                                         int accumulate, void *__restrict__ out,
                                                         const int64_t *__restrict__ offsets, int E, int64_t R) {
    const uint32_t per_group = static_cast<uint32_t>(n4) / static_cast<uint32_t>(E);
    const int e = threadIdx.x;  // E <= 256: bad offsets left the partial sums unwritten
    const bool bad = offsets && e < E && (offsets[e] < 0 || offsets[e + 1] < offsets[e] || offsets[e + 1] > R);
    if (__syncthreads_or(bad)) return;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n4; i += gridDim.x * 256ll) {
        if (TYPE == BEAM_MOE_F32 && accumulate && offsets) {
            const uint32_t g = static_cast<uint32_t>(i) / per_group;
            if (offsets[g + 1] == offsets[g]) continue;
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < splits; ++s) {
            const float4 v = __ldg(part + s * n4 + i);
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
        }
        if constexpr (TYPE == BEAM_MOE_F32) {
            float4 *o = reinterpret_cast<float4 *>(out) + i;
            if (accumulate) {
                const float4 v = *o;
                a.x += v.x;
                a.y += v.y;
                a.z += v.z;
                a.w += v.w;
            }
            *o = a;
        } else {
            reinterpret_cast<uint2 *>(out)[i] = make_uint2(pack2<TYPE>(a.x, a.y), pack2<TYPE>(a.z, a.w));
        }
    }
}

}  // namespace beam
