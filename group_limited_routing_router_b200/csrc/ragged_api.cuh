// Host side of the grouped products, the INT8 row quantisers and SwiGLU: argument checks, tensor maps,
// the choice of kernel, launches.  Follows beam_moe.cu in its translation unit (libbeam_moe.cu) and uses its
// device set-up and tensor-map encoder.
#pragma once

#include "ragged.cuh"
#include "swiglu.cuh"

namespace beam {
namespace {

// Split kernels: <BN, stages>.  A few rows per group: 32-row tiles in a 10-deep ring.  More rows but too few
// tiles for the pairs: 128-row tiles.
#define RS_FEW_ARGS 32, 10
#define RS_MID_ARGS 128, 5

struct RaggedDevice {
    std::once_flag once;
    int status = BEAM_MOE_OK;
    int pairs = 0, wgrad_pairs = 0;  // co-resident clusters of 2
    int clusters[4] = {0, 0, 0, 0};  // split kernels: co-resident clusters of 1, 2, 4, 8 CTAs
};
RaggedDevice g_ragged[kMaxDevices];

template <typename F>
int max_clusters(F *kernel, int threads, int smem, int size, int sms) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(size * (sms / size)), 1, 1);
    lc.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = static_cast<unsigned>(size);
    a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
    lc.attrs = a;
    lc.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &lc) != cudaSuccess) return 0;
    return std::min(n, sms / size);
}
template <typename F>
bool set_smem(F *kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}
template <int NA>
bool set_pair_smem() {
    constexpr int n = RpairCfg<NA>::kSmem;
    if constexpr (NA == 1)
        if (!set_smem(ragged_pair_kernel<true, false, NA>, n)) return false;
    return set_smem(ragged_pair_kernel<false, false, NA>, n) && set_smem(ragged_pair_kernel<false, true, NA>, n);
}
template <int BN, int ST>
bool set_split_smem() {
    constexpr int n = RsplitCfg<BN, ST>::kSmem;
    return set_smem(ragged_split_kernel<false, false, BN, ST>, n) &&
           set_smem(ragged_split_kernel<false, true, BN, ST>, n) &&
           set_smem(ragged_split_kernel<true, false, BN, ST>, n);
}

int init_ragged(int *dev_out) {
    int rc;
    if ((rc = init_device(dev_out))) return rc;
    RaggedDevice &d = g_ragged[*dev_out];
    const int sms = g_dev[*dev_out].num_sms;
    std::call_once(d.once, [&]() {
        bool ok = set_pair_smem<1>() && set_pair_smem<2>() && set_smem(ragged_wgrad_kernel<1>, RwgradCfg<1>::kSmem) &&
                  set_smem(ragged_wgrad_kernel<2>, RwgradCfg<2>::kSmem) &&
                  set_split_smem<RS_FEW_ARGS>() && set_split_smem<RS_MID_ARGS>();
        if (ok) {
            // one CTA per SM in all variants
            d.pairs = max_clusters(ragged_pair_kernel<false, false, 1>, kRgThreads, RpairCfg<1>::kSmem, 2, sms);
            d.wgrad_pairs = max_clusters(ragged_wgrad_kernel<1>, kRwThreads, RwgradCfg<1>::kSmem, 2, sms);
            for (int i = 0; i < 4; ++i)  // both split kernels run one CTA per SM
                d.clusters[i] = max_clusters(ragged_split_kernel<false, false, RS_MID_ARGS>, kRgThreads,
                                             RsplitCfg<RS_MID_ARGS>::kSmem, 1 << i, sms);
            ok = d.pairs > 0 && d.wgrad_pairs > 0 && d.clusters[0] > 0;
        }
        if (!ok) {
            cudaGetLastError();
            d.status = BEAM_MOE_ERR_CUDA;
        }
    });
    return d.status;
}

// Tensor maps of the operands: rows [rows][width] with a row stride, and weights / results [groups][rows][width].
bool map_rows(CUtensorMap *m, int esize, const void *base, uint64_t width, uint64_t ld, uint64_t rows, uint32_t box_w,
              uint32_t box_rows) {
    const CUtensorMapDataType dt = esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t dims[2] = {width, rows};
    const cuuint64_t strides[1] = {ld * static_cast<uint64_t>(esize)};
    const cuuint32_t box[2] = {box_w, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode_fn()(m, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_groups(CUtensorMap *m, CUtensorMapDataType dt, int esize, const void *base, uint64_t width, uint64_t rows,
                uint64_t groups, uint32_t box_w, uint32_t box_rows) {
    const cuuint64_t dims[3] = {width, rows, groups};
    const cuuint64_t strides[2] = {width * esize, width * rows * esize};
    const cuuint32_t box[3] = {box_w, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(m, dt, 3, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same rows as blocks of 64 16-bit columns [width / 64][rows][64] (width a multiple of 64), box 64 x 64 x 2:
// 128 columns of 64 rows in one load.
bool map_blocks(CUtensorMap *m, const void *base, uint64_t width, uint64_t ld, uint64_t rows) {
    const cuuint64_t dims[3] = {64, rows, width / 64};
    const cuuint64_t strides[2] = {ld * 2, 128};
    const cuuint32_t box[3] = {64, 64, 2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kMaxLd = int64_t(1) << 32;
int type_size(int t) { return t == BEAM_MOE_F32 ? 4 : 2; }
bool is16(int t) { return t == BEAM_MOE_BF16 || t == BEAM_MOE_F16; }
bool is_type(int t) { return is16(t) || t == BEAM_MOE_F32; }
// Width of a matrix: rows of whole 16-byte pieces.
bool width_ok(int64_t w, int step) { return w >= step && w <= 65536 && w % step == 0; }
// Row stride: at least the width, rows on 16-byte boundaries.
bool ld_ok(int64_t ld, int64_t width, int esize) { return ld >= width && ld <= kMaxLd && (ld * esize) % 16 == 0; }
bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// k-steps per accumulation segment.  Each instruction (16 products per sum; 4 to a k-step) truncates the
// running sum, half of 2^-23 of it on average, always toward zero: a sum that grows evenly loses 2^-25 of its
// end value per instruction, one of mixed signs far less (5120 products: 1.3e-6 in one segment, 2.3e-7 in
// segments of 256).  fp32 results: 4 k-steps, 2^-21.  16-bit results: 16 k-steps, 2^-19.
int segment_steps(bool i8, int out_type, int n_kb) {
    if (i8) return std::max(n_kb, 1);  // INT32 sums are exact
    return out_type == BEAM_MOE_F32 ? 4 : 16;
}
// The wide tiles sum 16-bit results in one segment where that loses at most an eighth of the result's half
// step: length / 16 x 2^-25 <= 2^-12 (bf16) or 2^-15 (fp16).
bool one_segment_ok(int dtype, int64_t length) { return length <= (dtype == BEAM_MOE_BF16 ? 131072 : 16384); }
// wgrad's wide tiles flush fp32 results every 4096 rows: 256 instructions, 2^-17 at most, against 2^-21 of the 256-column
// tiles.  Flushed every 1024 rows (2^-19) they are no faster than those (fp32, 8 groups of 8192 rows, 5120 x 2560: 1.51
// ms; every 1024 rows 1.82; 256-column tiles 1.86).
constexpr int kFlushSteps = 64;

uint32_t ragged_idesc(bool i8, int dtype, int M, bool a_mn, bool b_mn) {
    uint32_t d = static_cast<uint32_t>(M >> 4) << 24;
    if (i8) return d | (2u << 4) | (1u << 7) | (1u << 10);  // D int32, A and B signed 8-bit
    const uint32_t f = dtype == BEAM_MOE_BF16 ? 1u : 0u;    // A and B: 0 fp16, 1 bf16; D fp32
    return d | (1u << 4) | (f << 7) | (f << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16);
}

// A launch that the stream's last kernel need not have ended for: the kernel waits for it by itself (wait_for_stream).
// cluster: CTAs per cluster, 0 where the kernel says it.  One token, 5120 -> 20480, INT8 with its quantiser, calls
// back to back: 26.7 -> 22.5 us; SwiGLU and its gradient, 32768 x 2560: 191 -> 187; decode of 32 rows on 30 experts:
// 88 -> 86.
template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), dim3 grid, dim3 block, int smem, unsigned cluster, cudaStream_t s,
                 const A &...args) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = static_cast<size_t>(smem);
    lc.stream = s;
    cudaLaunchAttribute a[2];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    a[1].id = cudaLaunchAttributeClusterDimension;
    a[1].val.clusterDim.x = cluster;
    a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
    lc.attrs = a;
    lc.numAttrs = cluster ? 2 : 1;
    if (cudaLaunchKernelEx(&lc, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return BEAM_MOE_ERR_CUDA;
    }
    return launch_status();
}
template <bool I8, bool A_MN, int BN, int ST>
int launch_split(int S, int clusters, cudaStream_t s, const CUtensorMap &w, const CUtensorMap &b,
                 const RaggedParams &p) {
    return launch_after(ragged_split_kernel<I8, A_MN, BN, ST>, static_cast<unsigned>(S * clusters), kRgThreads,
                        RsplitCfg<BN, ST>::kSmem, static_cast<unsigned>(S), s, w, b, p);
}
template <int BN, int ST>
int launch_split_any(bool i8, bool a_mn, int S, int clusters, cudaStream_t s, const CUtensorMap &w,
                     const CUtensorMap &b, const RaggedParams &p) {
    if (i8) return launch_split<true, false, BN, ST>(S, clusters, s, w, b, p);
    if (a_mn) return launch_split<false, true, BN, ST>(S, clusters, s, w, b, p);
    return launch_split<false, false, BN, ST>(S, clusters, s, w, b, p);
}

template <bool I8, bool A_MN, int NA>
int launch_pair(int pairs, cudaStream_t s, const CUtensorMap &w, const RowMaps &b, const RaggedParams &p) {
    return launch_after(ragged_pair_kernel<I8, A_MN, NA>, static_cast<unsigned>(2 * pairs), kRgThreads,
                        RpairCfg<NA>::kSmem, 0, s, w, b, p);
}

// Kernel of a forward / dgrad product from its sizes alone (the counts stay on the device): rows spread
// over min(E, R) groups.
struct RaggedPlan {
    int pair;      // 256-feature tiles per CTA pair (1 or 2); 0: the split kernels
    bool few;      // split kernels: 32-row tiles
    int S, log_s;  // split kernels: CTAs per cluster
    int items;
};
// cut: rows that do not all start on 128-byte lines.
RaggedPlan ragged_plan(const RaggedDevice &d, int E, int64_t R, int M, int n_kb, bool wide_ok, bool cut) {
    RaggedPlan P{};
    const int64_t groups = std::min<int64_t>(E, R);
    const int64_t mean = (R + groups - 1) / groups;
    const int64_t row_tiles = groups * ((mean + kRpBN - 1) / kRpBN);
    const int64_t pair_items = row_tiles * ((M + kPairRows - 1) / kPairRows);
    P.few = mean <= 32;
    const int bn = P.few ? 32 : 128;
    // groups around the mean have half a row tile more than it fills, on average (16 of ~256 rows: 48 tiles, not 32)
    const int64_t halves =
        groups == 1 || 4 * mean <= 3 * bn ? 2 * ((mean + bn - 1) / bn) : (2 * mean + bn - 1) / bn + 1;
    const int64_t items = (groups * halves + 1) / 2 * ((M + kBM - 1) / kBM);
    int64_t best = 0;
    for (int i = 0; i < 4; ++i) {
        const int S = 1 << i;
        if (S > n_kb || d.clusters[i] == 0) break;
        // rounds over the co-resident clusters x (k-steps per CTA + the item's fixed cost in k-steps of ~0.37 us:
        // ~4, and for the exchange of the partial sums 1.2 us for 16 rows, 6 us for 128)
        const int64_t rows = std::min<int64_t>(mean, bn);
        const int64_t t = ((items + d.clusters[i] - 1) / d.clusters[i]) *
                          ((n_kb + S - 1) / S + 4 + (S > 1 ? rows / 8 : 0));
        if (i == 0 || t < best) {
            best = t;
            P.S = S;
            P.log_s = i;
        }
    }
    P.items = static_cast<int>(std::min<int64_t>(items, 1 << 30));
    if (P.few) return P;
    // Two feature tiles per pair where the rounds come out shorter.  Cycles per k-step of r rows: what L2
    // delivers, 1.4 per 64 bytes staged, half as much again where rows do not start on 128-byte lines; or the
    // products themselves, 2.75 r per 256 features under the power limit.  An item adds 2600 cycles, of two
    // tiles 7400 (the products wait for its epilogue), and takes as long as its results take to write, 6100 and
    // 15800; two tiles take half a round more, for uneven last rounds.  Measured, one tile against two: 8 groups of
    // 8192 rows, 5120 x 2560, 1174 / 1196 us; 32768 rows, 512 x 4096, 117 / 139; 56548 rows, 1000 x 1512
    // (lines cut), 182 / 153; 64 groups of ~256 rows (often two tiles of ~133), input gradient of 5120 x 2560,
    // 475 / 426; 256 of 128 rows, 5120 x 2560, 1345 / 1236; 16 of 256 rows, 2048 x 4096, 90 / 105; 8 of 950 rows,
    // 2728 x 4808 (cut), 213 / 188.
    const int64_t r = groups == 1 ? (mean + row_tiles - 1) / row_tiles : mean * kRpBN / (mean + kRpBN / 2);
    const int64_t tiles = groups == 1 ? row_tiles : (groups * mean + r - 1) / r;
    const int64_t rounds1 = (tiles * ((M + kPairRows - 1) / kPairRows) + d.pairs - 1) / d.pairs;
    const int64_t rounds2 = (tiles * ((M + 2 * kPairRows - 1) / (2 * kPairRows)) + d.pairs - 1) / d.pairs;
    const int64_t line = cut ? 9 : 6;
    const int64_t step1 = std::max((256 + r) * line * 11 / 48, r * 11 / 4);
    const int64_t step2 = std::max((512 + r) * line * 11 / 48, r * 11 / 2);
    const int64_t t1 = 2 * rounds1 * std::max<int64_t>(n_kb * step1 + 2600, 6100);
    const int64_t t2 = (2 * rounds2 + 1) * std::max<int64_t>(n_kb * step2 + 7400, 15800);
    // Fewer items than pairs go to the pairs where that is shorter by a tenth than splitting the contraction, by
    // the same cycles per k-step (split against pairs: 9312 rows in 4 groups, 5144 x 240, 82 / 47 us; 4096 rows,
    // 4096 x 1024, 53 / 35; 768 rows, 4096 x 4096, 51 / 33; 5000 rows in 32 groups, 2560 x 512, 45 / 31).
    const int64_t split = 2 * best * (256 + 2 * std::min<int64_t>(mean, 128)) * line * 11 / 48;
    if (pair_items < d.pairs && 10 * t1 > 9 * split) return P;
    P.pair = wide_ok && t2 < t1 && pair_items >= d.pairs ? 2 : 1;
    return P;
}

struct RaggedCall {
    bool i8, dgrad;
    int E;
    int64_t R;
    int K, N, dtype, out_type;
    const void *rows;  // x (forward) or dy (dgrad)
    int64_t ld_rows;
    const int64_t *offsets;
    const void *w;
    void *out;
    int64_t ldo;
    const float *row_scale, *channel_scale;
};

int ragged_product(const RaggedCall &c, cudaStream_t s) {
    const int step = c.i8 ? 16 : 8, esize = c.i8 ? 1 : 2;
    if (c.E < 1 || c.E > kPmMaxE || !width_ok(c.K, step) || !width_ok(c.N, step)) return BEAM_MOE_ERR_INVALID_CONFIG;
    if (!is_type(c.out_type) || (!c.i8 && (!is16(c.dtype) || (c.out_type != c.dtype && c.out_type != BEAM_MOE_F32))))
        return BEAM_MOE_ERR_INVALID_ARG;
    const int width = c.dgrad ? c.N : c.K, M = c.dgrad ? c.K : c.N;  // contraction, output features
    if (c.R < 0 || c.R > kMaxTokens || !ld_ok(c.ld_rows, width, esize) || !ld_ok(c.ldo, M, type_size(c.out_type)))
        return BEAM_MOE_ERR_INVALID_ARG;
    if (c.R == 0) return BEAM_MOE_OK;
    if (!c.rows || !c.w || !c.out || (!c.offsets && c.E != 1) || (c.i8 && (!c.row_scale || !c.channel_scale)))
        return BEAM_MOE_ERR_NULL;
    if (!aligned16(c.rows) || !aligned16(c.w) || !aligned16(c.out) || !aligned_to(c.offsets, 8) ||
        !aligned_to(c.row_scale, 4) || !aligned_to(c.channel_scale, 4))
        return BEAM_MOE_ERR_MISALIGNED;
    int dev, rc;
    if ((rc = init_ragged(&dev))) return rc;
    const RaggedDevice &d = g_ragged[dev];
    if (!encode_fn()) return BEAM_MOE_ERR_CUDA;
    const int kelems = kRgRowBytes / esize;
    const int n_kb = (width + kelems - 1) / kelems;
    const RaggedPlan P = ragged_plan(d, c.E, c.R, M, n_kb,
                                     !c.i8 && c.out_type != BEAM_MOE_F32 && one_segment_ok(c.dtype, width),
                                     (c.ld_rows | c.K) * esize % 128 != 0);
    RaggedParams p{};
    p.offsets = c.offsets;
    p.out = c.out;
    p.ldo = c.ldo;
    p.R = c.R;
    p.E = c.E;
    p.M = M;
    p.n_kb = n_kb;
    p.seg_kb = segment_steps(c.i8, c.out_type, n_kb);
    p.out_type = c.out_type;
    p.idesc = ragged_idesc(c.i8, c.dtype, P.pair ? kPairRows : kBM, c.dgrad, false);
    p.row_scale = c.row_scale;
    p.channel_scale = c.channel_scale;
    p.timeout = kDefaultTimeoutCycles;
    const uint32_t kbox = static_cast<uint32_t>(kelems);
    CUtensorMap m_w;
    // dgrad's weight tile is 64 features (K, contiguous) by 64 contraction rows (N), two boxes per 128 features
    if (!map_groups(&m_w, esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, esize, c.w,
                    c.K, c.N, c.E, kbox, c.dgrad ? 64 : kBM))
        return BEAM_MOE_ERR_CUDA;
    if (P.pair) {
        RowMaps m_b;
        for (int i = 0; i < kRpBoxes; ++i)
            if (!map_rows(&m_b.m[i], esize, c.rows, width, c.ld_rows, c.R, kbox,
                          static_cast<uint32_t>((i + 1) * kRpBoxStep)))
                return BEAM_MOE_ERR_CUDA;
        if (c.i8) return launch_pair<true, false, 1>(d.pairs, s, m_w, m_b, p);
        if (c.dgrad)
            return P.pair == 1 ? launch_pair<false, true, 1>(d.pairs, s, m_w, m_b, p)
                               : launch_pair<false, true, 2>(d.pairs, s, m_w, m_b, p);
        return P.pair == 1 ? launch_pair<false, false, 1>(d.pairs, s, m_w, m_b, p)
                           : launch_pair<false, false, 2>(d.pairs, s, m_w, m_b, p);
    }
    CUtensorMap m_b;
    if (!map_rows(&m_b, esize, c.rows, width, c.ld_rows, c.R, kbox,
                  P.few ? RsplitCfg<RS_FEW_ARGS>::kBox : RsplitCfg<RS_MID_ARGS>::kBox))
        return BEAM_MOE_ERR_CUDA;
    // items is an estimate where there are offsets: keep the whole GPU for uneven groups
    const int clusters = c.offsets ? d.clusters[P.log_s] : std::min(P.items, d.clusters[P.log_s]);
    return P.few ? launch_split_any<RS_FEW_ARGS>(c.i8, c.dgrad, P.S, clusters, s, m_w, m_b, p)
                 : launch_split_any<RS_MID_ARGS>(c.i8, c.dgrad, P.S, clusters, s, m_w, m_b, p);
}

// Splits of wgrad's rows: one where the result's tiles fill the 74 pairs of a 148-SM B200; else enough to
// fill them, of at least 512 rows of a mean group each.  The number of pairs is a constant, because the workspace's size
// is asked for without a device and has to be the same when the call is made; with other pairs the result is the same
// and only the time differs.
int wgrad_splits(int E, int64_t R, int K, int N) {
    const int64_t tiles = static_cast<int64_t>(E) * ((N + 255) / 256) * ((K + 255) / 256);
    const int64_t by_rows = R / E / 512;
    constexpr int64_t kSplitPairs = 74;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(kSplitPairs / tiles, by_rows), 64)));
}
// Whether wgrad's 256 x 512 tiles run: where their rounds come out shorter for a mean group, with the cycles
// measured per k-step (~690 for 256 columns, ~1060 for 512, both bound by L2) and per item (decoding and
// the hand-over; for 512 also its epilogue, which the products wait for).  bf16, 8 groups of 8192 rows: 1.17
// against 1.65 ms, 64 of 256: 0.44 against 0.49, 64 of 128: 0.44 against 0.37; fp32, 64 of 256: 0.87 against 0.79.
bool wgrad_wide(const RaggedDevice &d, int E, int64_t R, int K, int N, int splits, int dtype, int store) {
    if (splits > 1 || K <= 256 || (store != BEAM_MOE_F32 && !one_segment_ok(dtype, R))) return false;
    const int64_t n_kb = (R / E + 63) / 64, n_mt = (N + 255) / 256;
    const int64_t rounds1 = (E * n_mt * ((K + 255) / 256) + d.wgrad_pairs - 1) / d.wgrad_pairs;
    const int64_t rounds2 = (E * n_mt * ((K + 511) / 512) + d.wgrad_pairs - 1) / d.wgrad_pairs;
    const int64_t epilogue = store == BEAM_MOE_F32 ? 7000 * ((n_kb + kFlushSteps - 1) / kFlushSteps) : 2500;
    return rounds2 * (n_kb * 1060 + epilogue) < rounds1 * (n_kb * 690 + 700);
}
size_t wgrad_ws(int E, int64_t R, int K, int N) {
    const int s = R > 0 ? wgrad_splits(E, R, K, N) : 1;
    return s > 1 ? static_cast<size_t>(s) * E * N * K * 4 : 0;
}
bool wgrad_shape_ok(int E, int K, int N) { return E >= 1 && E <= kPmMaxE && width_ok(K, 8) && width_ok(N, 8); }

// Threads of the SwiGLU kernels: x covers eight columns each, up to 64 wide.
template <bool BACKWARD>
int launch_swiglu(int dtype, const SwigluParams &p, cudaStream_t s) {
    const int vecs = p.I / 8;
    int bx = 8;
    while (bx < 64 && bx < vecs) bx *= 2;
    const int by = 256 / bx;
    const int64_t gy = (p.R + by - 1) / by;
    const dim3 grid(static_cast<unsigned>((vecs + bx - 1) / bx), static_cast<unsigned>(std::min<int64_t>(gy, 65535)));
    const dim3 block(static_cast<unsigned>(bx), static_cast<unsigned>(by));
    if (dtype == BEAM_MOE_BF16) return launch_after(swiglu_kernel<__nv_bfloat16, BACKWARD>, grid, block, 0, 0, s, p);
    if (dtype == BEAM_MOE_F16) return launch_after(swiglu_kernel<__half, BACKWARD>, grid, block, 0, 0, s, p);
    return launch_after(swiglu_kernel<float, BACKWARD>, grid, block, 0, 0, s, p);
}

template <typename T, bool SWIGLU>
int launch_quant_t(const QuantParams &p, cudaStream_t s) {
    constexpr int kSteps = kQuantCached;
    const int vecs = p.K / 8;
    if (vecs <= 32 * kSteps)
        return launch_after(quant_i8_kernel<T, SWIGLU, true>, static_cast<unsigned>((p.R + 7) / 8), 256, 0, 0, s, p);
    const int threads = std::min(512, ((vecs + kSteps - 1) / kSteps + 31) / 32 * 32);
    return launch_after(quant_i8_kernel<T, SWIGLU, false>, static_cast<unsigned>(p.R), static_cast<unsigned>(threads),
                        0, 0, s, p);
}
template <bool SWIGLU>
int launch_quant(int dtype, const QuantParams &p, cudaStream_t s) {
    if (dtype == BEAM_MOE_BF16) return launch_quant_t<__nv_bfloat16, SWIGLU>(p, s);
    if (dtype == BEAM_MOE_F16) return launch_quant_t<__half, SWIGLU>(p, s);
    return launch_quant_t<float, SWIGLU>(p, s);
}

int rows_check(int64_t R, int I, int dtype) {
    if (!width_ok(I, 8)) return BEAM_MOE_ERR_INVALID_CONFIG;
    if (R < 0 || R > kMaxTokens || !is_type(dtype)) return BEAM_MOE_ERR_INVALID_ARG;
    return BEAM_MOE_OK;
}

}  // namespace
}  // namespace beam

extern "C" {

int beam_moe_grouped_mm(int32_t n_experts, int64_t R, int32_t K, int32_t N, int dtype, const void *x, int64_t ldx,
                        const int64_t *offsets, const void *w, int out_dtype, void *out, int64_t ldo, void *stream) {
    return beam::ragged_product({false, false, n_experts, R, K, N, dtype, out_dtype, x, ldx, offsets, w, out, ldo,
                                 nullptr, nullptr},
                                static_cast<cudaStream_t>(stream));
}

int beam_moe_grouped_mm_dgrad(int32_t n_experts, int64_t R, int32_t K, int32_t N, int dtype, const void *dy,
                              int64_t ldy, const int64_t *offsets, const void *w, int out_dtype, void *dx, int64_t ldx,
                              void *stream) {
    return beam::ragged_product({false, true, n_experts, R, K, N, dtype, out_dtype, dy, ldy, offsets, w, dx, ldx,
                                 nullptr, nullptr},
                                static_cast<cudaStream_t>(stream));
}

int beam_moe_grouped_mm_i8(int32_t n_experts, int64_t R, int32_t K, int32_t N, const int8_t *q, const float *row_scale,
                           const int64_t *offsets, const int8_t *w, const float *channel_scale, int out_dtype,
                           void *out, int64_t ldo, void *stream) {
    return beam::ragged_product({true, false, n_experts, R, K, N, BEAM_MOE_BF16, out_dtype, q, K, offsets, w, out, ldo,
                                 row_scale, channel_scale},
                                static_cast<cudaStream_t>(stream));
}

size_t beam_moe_grouped_mm_wgrad_workspace_size(int32_t n_experts, int64_t R, int32_t K, int32_t N) {
    if (!beam::wgrad_shape_ok(n_experts, K, N) || R < 0 || R > beam::kMaxTokens) return 0;
    return beam::wgrad_ws(n_experts, R, K, N);
}

int beam_moe_grouped_mm_wgrad(int32_t n_experts, int64_t R, int32_t K, int32_t N, int dtype, const void *dy,
                              int64_t ldy, const void *x, int64_t ldx, const int64_t *offsets, int out_dtype, void *dw,
                              int accumulate, void *ws, size_t ws_bytes, void *stream) {
    using namespace beam;
    if (!wgrad_shape_ok(n_experts, K, N)) return BEAM_MOE_ERR_INVALID_CONFIG;
    if (!is16(dtype) || (out_dtype != dtype && out_dtype != BEAM_MOE_F32) || R < 0 || R > kMaxTokens ||
        !ld_ok(ldy, N, 2) || !ld_ok(ldx, K, 2) || (accumulate && out_dtype != BEAM_MOE_F32))
        return BEAM_MOE_ERR_INVALID_ARG;
    if (!dw) return BEAM_MOE_ERR_NULL;
    if (!aligned16(dw)) return BEAM_MOE_ERR_MISALIGNED;
    if (R > 0) {
        if (!dy || !x || (!offsets && n_experts != 1)) return BEAM_MOE_ERR_NULL;
        if (!aligned16(dy) || !aligned16(x) || !aligned_to(offsets, 8)) return BEAM_MOE_ERR_MISALIGNED;
    }
    const size_t need = wgrad_ws(n_experts, R, K, N);
    if (need) {
        if (!ws) return BEAM_MOE_ERR_NULL;
        if (!aligned16(ws)) return BEAM_MOE_ERR_MISALIGNED;
        if (ws_bytes < need) return BEAM_MOE_ERR_WORKSPACE_TOO_SMALL;
    }
    int dev, rc;
    if ((rc = init_ragged(&dev))) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t n = static_cast<int64_t>(n_experts) * N * K;
    if (R == 0) {
        if (!accumulate && cudaMemsetAsync(dw, 0, static_cast<size_t>(n) * type_size(out_dtype), s) != cudaSuccess) {
            cudaGetLastError();
            return BEAM_MOE_ERR_CUDA;
        }
        return BEAM_MOE_OK;
    }
    if (!encode_fn()) return BEAM_MOE_ERR_CUDA;
    const int splits = wgrad_splits(n_experts, R, K, N);
    const int store = splits > 1 ? BEAM_MOE_F32 : out_dtype;
    WgradParams p{};
    p.g.offsets = offsets;
    p.g.R = R;
    p.g.E = n_experts;
    p.g.M = N;
    const bool wide = wgrad_wide(g_ragged[dev], n_experts, R, K, N, splits, dtype, store);
    // NB = 2: 16-bit results in one segment, fp32 ones flushed
    p.g.seg_kb = !wide ? segment_steps(false, store, 0) : (store == BEAM_MOE_F32 ? kFlushSteps : 1 << 30);
    p.g.out_type = store;
    p.g.idesc = ragged_idesc(false, dtype, kPairRows, true, true);
    p.g.timeout = kDefaultTimeoutCycles;
    p.K = K;
    p.n_mt = (N + 255) / 256;
    p.n_nt = wide ? (K + 511) / 512 : (K + 255) / 256;
    p.nt_inv = static_cast<uint32_t>(((uint64_t(1) << 32) + p.n_nt - 1) / p.n_nt);  // n_nt = 1 is not divided by
    p.splits = splits;
    p.accumulate = splits > 1 ? 0 : (accumulate != 0);
    const CUtensorMapDataType dt = store == BEAM_MOE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                         : (store == BEAM_MOE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
    CUtensorMap m_dy, m_x, m_dw;
    p.dy_blocks = N % 64 == 0;
    p.x_blocks = K % 64 == 0;
    if (!(p.dy_blocks ? map_blocks(&m_dy, dy, N, ldy, R) : map_rows(&m_dy, 2, dy, N, ldy, R, 64, 64)) ||
        !(p.x_blocks ? map_blocks(&m_x, x, K, ldx, R) : map_rows(&m_x, 2, x, K, ldx, R, 64, 64)) ||
        !map_groups(&m_dw, dt, type_size(store), splits > 1 ? ws : dw, K, N, static_cast<uint64_t>(splits) * n_experts,
                    128u / static_cast<uint32_t>(type_size(store)), 32))
        return BEAM_MOE_ERR_CUDA;
    const unsigned wg = static_cast<unsigned>(2 * g_ragged[dev].wgrad_pairs);
    rc = wide ? launch_after(ragged_wgrad_kernel<2>, wg, kRwThreads, RwgradCfg<2>::kSmem, 0, s, m_dy, m_x, m_dw, p)
              : launch_after(ragged_wgrad_kernel<1>, wg, kRwThreads, RwgradCfg<1>::kSmem, 0, s, m_dy, m_x, m_dw, p);
    if (rc || splits == 1) return rc;
    const int64_t n4 = n / 4;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((n4 + 255) / 256, 8 * g_dev[dev].num_sms));
    const float4 *part = static_cast<const float4 *>(ws);
    if (out_dtype == BEAM_MOE_BF16)
        ragged_join_kernel<BEAM_MOE_BF16><<<grid, 256, 0, s>>>(part, splits, n4, 0, dw, offsets, n_experts, R);
    else if (out_dtype == BEAM_MOE_F16)
        ragged_join_kernel<BEAM_MOE_F16><<<grid, 256, 0, s>>>(part, splits, n4, 0, dw, offsets, n_experts, R);
    else
        ragged_join_kernel<BEAM_MOE_F32>
            <<<grid, 256, 0, s>>>(part, splits, n4, accumulate != 0, dw, offsets, n_experts, R);
    return launch_status();
}

int beam_moe_quant_i8_rows(int64_t R, int32_t K, int dtype, const void *x, int64_t ldx, int8_t *q, float *scale,
                           void *stream) {
    using namespace beam;
    int rc = rows_check(R, K, dtype);
    if (rc) return rc;
    if (!ld_ok(ldx, K, type_size(dtype))) return BEAM_MOE_ERR_INVALID_ARG;
    if (R == 0) return BEAM_MOE_OK;
    if (!x || !q || !scale) return BEAM_MOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned_to(scale, 4)) return BEAM_MOE_ERR_MISALIGNED;
    int dev;
    if ((rc = init_device(&dev))) return rc;
    return launch_quant<false>(dtype, QuantParams{x, nullptr, ldx, 0, q, scale, R, K},
                               static_cast<cudaStream_t>(stream));
}

int beam_moe_swiglu_i8(int64_t R, int32_t I, int dtype, const void *g, int64_t ldg, const void *u, int64_t ldu,
                       int8_t *q, float *scale, void *stream) {
    using namespace beam;
    int rc = rows_check(R, I, dtype);
    if (rc) return rc;
    if (!ld_ok(ldg, I, type_size(dtype)) || !ld_ok(ldu, I, type_size(dtype))) return BEAM_MOE_ERR_INVALID_ARG;
    if (R == 0) return BEAM_MOE_OK;
    if (!g || !u || !q || !scale) return BEAM_MOE_ERR_NULL;
    if (!aligned16(g) || !aligned16(u) || !aligned16(q) || !aligned_to(scale, 4)) return BEAM_MOE_ERR_MISALIGNED;
    int dev;
    if ((rc = init_device(&dev))) return rc;
    return launch_quant<true>(dtype, QuantParams{g, u, ldg, ldu, q, scale, R, I},
                              static_cast<cudaStream_t>(stream));
}

int beam_moe_swiglu(int64_t R, int32_t I, int dtype, const void *g, int64_t ldg, const void *u, int64_t ldu, void *h,
                    int64_t ldh, void *stream) {
    using namespace beam;
    int rc = rows_check(R, I, dtype);
    if (rc) return rc;
    const int es = type_size(dtype);
    if (!ld_ok(ldg, I, es) || !ld_ok(ldu, I, es) || !ld_ok(ldh, I, es)) return BEAM_MOE_ERR_INVALID_ARG;
    if (R == 0) return BEAM_MOE_OK;
    if (!g || !u || !h) return BEAM_MOE_ERR_NULL;
    if (!aligned16(g) || !aligned16(u) || !aligned16(h)) return BEAM_MOE_ERR_MISALIGNED;
    int dev;
    if ((rc = init_device(&dev))) return rc;
    SwigluParams p{};
    p.g = g, p.u = u, p.h = h;
    p.ld_g = ldg, p.ld_u = ldu, p.ld_h = ldh;
    p.R = R, p.I = I;
    return launch_swiglu<false>(dtype, p, static_cast<cudaStream_t>(stream));
}

int beam_moe_swiglu_backward(int64_t R, int32_t I, int dtype, const void *dh, int64_t lddh, const void *g, int64_t ldg,
                             const void *u, int64_t ldu, void *dg, int64_t lddg, void *du, int64_t lddu, void *stream) {
    using namespace beam;
    int rc = rows_check(R, I, dtype);
    if (rc) return rc;
    const int es = type_size(dtype);
    if (!ld_ok(lddh, I, es) || !ld_ok(ldg, I, es) || !ld_ok(ldu, I, es) || !ld_ok(lddg, I, es) || !ld_ok(lddu, I, es))
        return BEAM_MOE_ERR_INVALID_ARG;
    if (R == 0) return BEAM_MOE_OK;
    if (!dh || !g || !u || !dg || !du) return BEAM_MOE_ERR_NULL;
    if (!aligned16(dh) || !aligned16(g) || !aligned16(u) || !aligned16(dg) || !aligned16(du))
        return BEAM_MOE_ERR_MISALIGNED;
    int dev;
    if ((rc = init_device(&dev))) return rc;
    SwigluParams p{};
    p.dh = dh, p.g = g, p.u = u, p.dg = dg, p.du = du;
    p.ld_dh = lddh, p.ld_g = ldg, p.ld_u = ldu, p.ld_dg = lddg, p.ld_du = lddu;
    p.R = R, p.I = I;
    return launch_swiglu<true>(dtype, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
