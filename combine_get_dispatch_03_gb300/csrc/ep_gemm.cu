// ep_gemm.cu -- matrix products grouped by expert, with ragged groups (sm_103a tensor cores).
//
// Rows of all experts lie in one array; expert e has rows [begin[e], begin[e] + count[e]) and its own
// weights.  Its kernels are of one template:
//   forward       out[r][j] = sum_c x[r][c] * w[e][j][c]          bf16, both operands contraction-major
//   transposed    out[r][j] = sum_c x[r][c] * w[e][c][j]          bf16, the weights read across (gradient of the rows)
//   weight grad   dw[e][j][c] = sum_r dy[r][j] * x[r][c]          bf16, both operands read across, over a group's rows
//   fp8           out[r][j] = sum_b sx[r][b] * sw[e][j/128][b] * sum_{c in b} x[r][c] * w[e][j][c]    e4m3, blocks b of 128
// and the forward form with an epilogue (finish_columns()), v = x w^T + bias:
//   activated     out[r][j] = act(v[r][j]) * row_weights[r] + residual[r][j]
//   gated         out[r][j] = act(v[r][j]) * v[r][width + j] * row_weights[r] + residual[r][j]
// A gated tile's columns are half gate, half up: both accumulators of an output lie in the same lane of tensor memory.
//
// Work is cut into output tiles of 128 rows (256 for a pair of CTAs) by 64, 128 or 256 columns, taken
// in turn by the CTAs of one resident wave.  In a CTA one thread loads operand tiles with tensor maps into a
// ring of shared-memory stages (128 bytes of the contraction a stage), one thread issues tcgen05.mma from
// them into tensor memory, and eight warps read the fp32 accumulators back, round and store.  Two
// accumulators of 256 columns let the next tile's products run under this tile's stores.
//
// What bounds it, measured on a GB300 (1946.7 TFLOP/s bf16, 6787 GB/s copied):
//   - many rows an expert, bf16: the tensor cores, at the clock that the power limit leaves, so that times go by the card
//     and by how long it has been busy.  8 experts of 2048 rows, 4096 x 7168: 521 to 549 us, 1750 to 1850 TFLOP/s, 512
//     to 516 cycles a stage where a stage's products take 512; the gradient of the rows 510 to 572 us, of the weights
//     557 to 639 us (its 0.94 GB of fp32 results and the ends of groups cost the rest; 573 to 591 in bf16).
//   - few rows an expert: memory, the weights.  32 experts of 64 rows, 4096 x 7168 bf16: 286 to 309 us, 6.2 to 6.7 TB/s.
//   - FP8: a block's sums go from tensor memory through registers, 32768 FMAs a stage and CTA at 128 a cycle; with the
//     way there and back between the products' thread and the eight warps a stage takes about 770 cycles for
//     512 of products.  The same 8 experts: 340 to 362 us, 2660 to 2820 TFLOP/s; 64 experts of 128 rows read from
//     messages: 308 to 334 us, 6.0 to 6.5 TB/s (375 to 385 where half of the experts have more than 128).
//   - short contractions and few rows: the results' way out (staged_pays()).  64 experts of 1024 rows, 4096 x 256 bf16:
//     128 to 138 us, 5.1 to 5.5 TB/s; gradients of 32 experts of 16 rows, 2048 x 2048: 89 us, 6.0 TB/s.
//   - few tiles: a launch, the table of groups (2000 cycles), and 250 to 400 cycles a step however little it computes
//     (deep_stages()): 16 rows, 1024 x 7168 19.3 us; with an epilogue and a workspace in eight parts 10.2.
//   - an epilogue: 8187 rows, 7168 x 2048 121 us without anything (120 without the form), 125 with a bias, 144 with a residual (117 MB
//     more), 149 with gelu, 146 with silu, 139 gated: where a tile's contraction is short, its eight warps do not keep up.
//   - rows four bytes apart: the two warps that copy them, a round trip to memory for every 8 or 16 rows (copy_rows()).
//
// Two loads of 16 KB a stage (one an operand) rather than smaller ones: a load costs the issuing thread about
// 95 cycles.  64 columns of an accumulator a read in the FP8 form: 292 cycles for 128 columns and their FMAs in eight
// warps, 335 with 32 a read.
//
// The group table (tiles before each expert, counts, begins) is built in shared memory by each CTA from the
// device arrays, so that no count has to reach the host.
#include <cudaTypedefs.h>

#include "ep_act.cuh"
#include "ep_groups.cuh"
#include "ep_handle.h"
#include "ep_maps.h"
#include "ep_tc.cuh"
#include "ep_trace.h"

namespace ep {

// The driver's tensor-map encoder, looked up once (the library does not link against libcuda).
static PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

ep_status encode(CUtensorMap* map, const Operand& o) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = map_encoder();
    if (fn == nullptr) return fail(EP_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    cuuint64_t size[4], stride[3];
    cuuint32_t box[4], step[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) size[i] = o.size[i], box[i] = o.box[i];
    for (int i = 0; i < 3; ++i) stride[i] = o.stride[i];
    const CUtensorMapDataType type = o.element == Element::kFp8    ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : o.element == Element::kFp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUresult rc = CUDA_SUCCESS;
    for (int attempt = 0; attempt < 2; ++attempt) {
        rc = fn(map, type, o.dims, const_cast<void*>(o.base), size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (rc != CUDA_ERROR_INVALID_CONTEXT) break;
        // A thread that has not used its device yet has no context, and the encoder, unlike the runtime's calls, makes
        // none current.
        int device = 0;
        cudaError_t err = cudaGetDevice(&device);
        if (err == cudaSuccess) err = cudaSetDevice(device);
        if (err != cudaSuccess) return cuda_fail(err, "making the device's context current");
    }
    if (rc != CUDA_SUCCESS) return fail(EP_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(rc));
    return EP_OK;
}

namespace {

enum GemmForm { kForward = 0, kTransposed = 1, kWeightGrad = 2, kFp8 = 3, kActivated = 4, kGated = 5, kActivatedFp32 = 6 };
constexpr bool has_epilogue(int form) { return form >= kActivated; }

// Steps (128 bytes of the contraction) that one accumulator sums in tensor memory before its sums are added up in
// fp32 registers; 0: all of them.  FP8: one block, for its scales.  Weight gradient: 512 rows -- the tensor cores cut
// sums off instead of rounding them, and 2048 rows in one accumulator left 1.9e-6 of the result against 64 bits, 768
// 6.7e-7, 640 5.8e-7, 512 4.7e-7 (the same sums of products in fp32 by a library: 3.9e-7), for 1113 (768), 1164 and 1179 us
// at 65536 rows, 32 experts of 2048 x 7168, and 1125 us where they leave through shared memory (staged_pays()).  The
// activated form's fp32 output (a router's logits) is summed like it: over 7168 in one accumulator it was off by 7.9e-6.  The
// other forms round to bf16, far above that.
constexpr int segment_steps(int form) { return form == kFp8 ? 1 : form == kWeightGrad || form == kActivatedFp32 ? 8 : 0; }

constexpr int kTileRows = 128;      // output rows per CTA
constexpr int kMaxTileCols = 256;
constexpr int kRowBytes = 128;      // bytes of one operand row in a stage (the swizzle's span)
constexpr int kBox = 128;           // output elements (rows or columns) of a tensor-map load: 16 KB
constexpr int kRowBox = 32;         // the same for a group's last rows: a short group loads few
constexpr int kColBox = 64;         // the same for narrow tiles
constexpr int kPairRowsFp8 = 1024;  // rows of a group from which the FP8 form runs on pairs of CTAs
constexpr int kMaxStages = 12;
constexpr int kEpilogueWarps = 8;
constexpr int kGemmThreads = (4 + kEpilogueWarps) * kWarpSize;  // warps 0 to 3 for loads and products: registers go by four warps
constexpr int kControlBytes = 704;  // static shared memory
constexpr int kLeastPartSteps = 8;
constexpr int kMostParts = 8;
constexpr int kPartFloats = 128 * kWarpSize;  // a warp's sums of a part: 128 columns at most
constexpr uint32_t kOutBox = 32 * kRowBytes;  // a warp's results on their way out: 32 rows of 128 bytes
// Of them a warp: in FP8 one for each 64 columns, since there a tile's stores hold up the next one's sums (2048 rows an
// expert, 7168 x 2048: 1740 us with one, 1682 with two).
constexpr int out_boxes(int form) { return form == kFp8 ? 2 : 1; }
constexpr int kMaxSmem = 232448 - kControlBytes;

struct GemmParams {
    Groups groups;          // of the row operand (weight grad: operands) and the output's rows
    int32_t rows_dim;       // weight grad: output rows per group (n)
    int32_t cols_dim;       // output columns
    int32_t contraction;    // contraction length (weight grad: a group's count instead)
    void* out;
    int64_t out_row_bytes;
    const uint8_t* x_scales;
    int64_t x_scale_row_bytes;
    const float* w_scales;
    int32_t scales_ue8m0;
    int32_t out_fp32;       // weight grad: then staged
    int32_t accumulate;     // weight grad
    int32_t wide_stores;    // output rows are 32-byte aligned
    int32_t tile_overhead;  // columns that a tile's width-independent cost is worth
    int32_t staged;         // blocks of 32 rows go out through shared memory
    int32_t a_chunked, b_chunked;  // operands read across: columns up to which loads of kBox reach (then kColBox)
    const uint8_t* a_words;        // rows that no tensor map can describe (not 16 bytes apart), or NULL
    int64_t a_row_bytes;
    int32_t* status;
    uint64_t wait_limit_ns;
    // the epilogue of the forms that have one; each may be NULL
    const float* bias;          // [groups][n]
    const float* row_weights;   // [num_rows]
    const uint8_t* residual;    // bf16 rows like the output's
    int64_t residual_row_bytes;
    uint8_t* pre;               // v in bf16, rows of n
    int64_t pre_row_bytes;
    int32_t pre_wide;           // its rows are 32-byte aligned
    int32_t act;
    float* parts;               // where parts of a contraction meet: [tile][part][warp][column][lane], or NULL: it is not cut
    int32_t* tickets;           // [tile][warp], 0
};

// Tensor maps of the two operands: loads of kBox output elements, and smaller ones; and of the results, boxes of 32
// rows by 128 bytes, as of the residual.
struct Maps {
    CUtensorMap a, a_small, b, b_small, out, residual;
};

// Where a warp's 32 rows of a tile go: the output row of the first (weight grad: in the group), how many of them exist,
// the first column.
struct alignas(16) Place {
    int row, col, group;
    short rows, cols;
};
static_assert(sizeof(Place) == 16 && alignof(Place) == 16, "read as one vector");

// Read where it is used (a plain read could be made early and kept in registers).
__device__ __forceinline__ Place read_place(const Place* from) {
    int4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem_u32(from)) : "memory");
    return {v.x, v.y, v.z, static_cast<short>(v.w & 0xffff), static_cast<short>(v.w >> 16)};
}

struct Control {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t tail_full[kMaxStages];  // weight grad: instead of full, for a group's last, partial block of rows; epilogue: a warp's residual
    uint64_t drained;  // every product has been computed
    uint32_t tmem;
    int32_t abort_flag;
    int64_t warp_sums[kGemmThreads / kWarpSize];
    int64_t warp_rows[kGemmThreads / kWarpSize];
    int32_t tiles, col_tiles, tile_cols;  // output tiles in all (parts of them), tiles across, columns of one
    int32_t parts, part_steps;            // of a tile's contraction, and steps of one
    Place at[kEpilogueWarps];             // forms with segments: of the tile that a warp is adding up
};
static_assert(sizeof(Control) <= kControlBytes, "control block");

struct Tile {
    int group, row0, rows, m0, n0, cols, steps;  // rows: valid rows of the group; m0: tile's first row in the group
    int step0, tile;                             // parts: the first step, the tile
};

// Steps of a stage.  A step's commit takes its 380 cycles whether one product lies before it or four, so that the narrowest tiles of
// single CTAs have two steps a stage and a commit (16 rows, 1024 x 7168: 26.5 to 19.3 us).  Tiles of 128 columns do not: three
// stages of 64 KB instead of six of 32 keep too little on its way (4096 rows, 256 x 7168: 24.9 to 27.1).
template <int FORM, int CG, bool kWords>
__device__ __forceinline__ bool deep_stages(int tile_cols) {
    return CG == 1 && !kWords && (FORM == kForward || has_epilogue(FORM)) && tile_cols <= kColBox;
}

// The group table in shared memory.
struct Table {
    int32_t* before;  // [groups + 1] row tiles before each group
    int32_t* count;   // [groups]
    int32_t* begin;   // [groups]
};

// Output columns of a tile of `cols` columns of products, and the fewest columns of products.
template <int FORM>
__device__ __forceinline__ int out_cols(int cols) { return FORM == kGated ? cols / 2 : cols; }
template <int FORM, int CG>
constexpr int min_cols() { return kColBox * (FORM == kGated ? 2 : CG); }

template <int FORM, int CG>
__device__ __forceinline__ Tile decode(const Table& t, const GemmParams& p, const Control& ctl, int tile) {
    Tile r;
    int part = 0;
    if constexpr (has_epilogue(FORM)) {
        if (ctl.parts > 1) {
            part = static_cast<uint32_t>(tile) % ctl.parts;
            tile = static_cast<uint32_t>(tile) / ctl.parts;
        }
    }
    r.tile = tile;
    const int lo = find_group(t.before, p.groups.groups, tile / ctl.col_tiles);
    const int in = tile - t.before[lo] * ctl.col_tiles;
    const int row_tiles = t.before[lo + 1] - t.before[lo];
    r.group = lo;
    r.row0 = t.begin[lo];
    r.rows = t.count[lo];
    // row tiles turn fastest: CTAs side by side share a weight tile
    r.n0 = in / row_tiles * out_cols<FORM>(ctl.tile_cols);
    // the last tile across is no wider than it has to be
    r.cols = ctl.tile_cols;
    while (r.cols > min_cols<FORM, CG>() && 2 * (p.cols_dim - r.n0) <= out_cols<FORM>(r.cols)) r.cols >>= 1;
    r.m0 = in % row_tiles * (kTileRows * CG);
    if constexpr (FORM == kWeightGrad) r.steps = (r.rows + 63) >> 6;
    else if constexpr (FORM == kFp8) r.steps = (p.contraction + 127) >> 7;
    else r.steps = (p.contraction + 63) >> 6;
    r.step0 = 0;
    if constexpr (has_epilogue(FORM)) {
        r.step0 = part * ctl.part_steps;
        r.steps = min(ctl.part_steps, r.steps - r.step0);
    }
    return r;
}

// Fills the table: clamps every group to the rows that exist (the first group that does not fit sets
// EP_ERR_CAPACITY), and sums the row tiles and, where rows are written, the rows.  All threads of the CTA.
template <int FORM, int CG>
__device__ __forceinline__ void build_table(const Table& t, const GemmParams& p, Control& ctl) {
    constexpr int kRows = kTileRows * CG;
    const int groups = p.groups.groups;
    const int per = (groups + kGemmThreads - 1) / kGemmThreads;
    const int first = threadIdx.x * per;
    const int last = min(first + per, groups);
    int64_t sum = 0, row_tiles = 0, rows = 0;
    for (int g = first; g < last; ++g) {
        const Group q = load_group(p.groups, g, p.status);
        rows += q.count;
        t.count[g] = q.count;
        t.begin[g] = q.begin;
        t.before[g] = static_cast<int32_t>(sum);
        sum += (static_cast<int64_t>(FORM == kWeightGrad ? p.rows_dim : q.count) + kRows - 1) / kRows;
    }
    if constexpr (FORM != kWeightGrad) {
#pragma unroll
        for (int o = kWarpSize / 2; o > 0; o >>= 1) rows += __shfl_xor_sync(kFullMask, rows, o);
        if (lane_id() == 0) ctl.warp_rows[threadIdx.x / kWarpSize] = rows;  // read after the prefix's barrier
    }
    const int64_t base = block_prefix<kGemmThreads>(sum, ctl.warp_sums, &row_tiles);
    for (int g = first; g < last; ++g) t.before[g] += static_cast<int32_t>(base);
    if (threadIdx.x < kWarpSize) {
        // Groups that together hold more rows than there are overlap: nothing is computed.  The rows decide, not the
        // tiles: eight groups of the same 100 rows have no more tiles than eight groups of 100 rows apart.
        bool overlap = false;
        if constexpr (FORM != kWeightGrad) {
            rows = 0;
            for (int w = 0; w < kGemmThreads / kWarpSize; ++w) rows += ctl.warp_rows[w];
            overlap = rows > p.groups.num_rows;
        }
        const int total = overlap ? 0 : static_cast<int>(row_tiles);
        // Tile width: the one whose waves over the CTAs take the least time, a wave costing its columns plus
        // what a tile costs at any width.  With an epilogue, few tiles and a workspace also parts of the contraction, one
        // wave of them.  A step of a column is worth 1.65 cycles (64 columns of few rows take 270 a step, 128 380, 256 650);
        // the parts' way out took 16 cycles a column, their way back to the last CTA 10 to 15 a column and part (4096 rows, 256 x
        // 7168: 25 us with two parts of 128 columns, 28 with four of 256).  A lane has a width and a number of parts: one thread
        // took 4 us over all of them while the others waited (16 rows, 1024 x 7168: 16.8 us a call, 13.0 by lanes).
        // (In 32 bits: there are fewer than 2^30 tiles.)
        static_assert(kWarpSize / kMostParts >= 4, "a lane for each");
        const int step = lane_id() / kMostParts, cols = kMaxTileCols >> step, parts = lane_id() % kMostParts + 1;
        const int shift = 8 - step - (FORM == kGated);  // of the columns of an output tile
        const uint32_t workers = gridDim.x / CG, steps = (p.contraction + 63) >> 6;
        const uint32_t across = static_cast<uint32_t>(p.cols_dim + (1 << shift) - 1) >> shift, tiles = total * across;
        uint32_t part_steps = steps;
        uint64_t cost = UINT64_MAX;
        if (cols >= min_cols<FORM, CG>()) {
            const uint32_t each = cols + (has_epilogue(FORM) ? max(p.tile_overhead, 100) : p.tile_overhead);
            if (parts == 1) {
                cost = static_cast<uint64_t>((tiles + workers - 1) / workers) * each * (has_epilogue(FORM) ? steps : 1);
            } else if (has_epilogue(FORM) && p.parts && tiles != 0 && tiles <= workers && parts * tiles <= workers && static_cast<uint32_t>(parts) * kLeastPartSteps <= steps) {
                part_steps = (steps + parts - 1) / parts;
                cost = static_cast<uint64_t>(part_steps) * each + 1000 + cols * (8 + 6 * parts);
            }
        }
        // the first of the cheapest
        const uint32_t high = static_cast<uint32_t>(cost >> 32), least = __reduce_min_sync(kFullMask, high);
        const uint32_t low = high == least ? static_cast<uint32_t>(cost) : UINT32_MAX;
        const uint32_t least_low = __reduce_min_sync(kFullMask, low);  // by all lanes
        if (lane_id() == __ffs(__ballot_sync(kFullMask, high == least && low == least_low)) - 1) {
            if (overlap) report(p.status, EP_ERR_CAPACITY);
            t.before[groups] = total;
            ctl.tile_cols = cols;
            ctl.col_tiles = across;
            ctl.part_steps = part_steps;
            ctl.parts = parts == 1 ? 1 : (steps + part_steps - 1) / part_steps;
            ctl.tiles = tiles * ctl.parts;
        }
    }
}

// A row's scale of one block as it lies in memory, and as the fp32 it stands for.
__device__ __forceinline__ uint32_t raw_scale(const uint8_t* row, int block, int ue8m0) {
    return ue8m0 ? row[block] : *reinterpret_cast<const uint32_t*>(row + 4 * static_cast<int64_t>(block));
}

__device__ __forceinline__ float scale_value(uint32_t raw, int ue8m0) {
    if (!ue8m0) return __uint_as_float(raw);
    return __uint_as_float(raw == 255 ? 0x7fc00000u : raw == 0 ? 0x00400000u : raw << 23);
}

// 32 columns of one output row, rounded to bf16; columns at or past `cols` (a multiple of 8) are left out.
__device__ __forceinline__ void store_bf16(uint8_t* row, int col, int cols, const float (&v)[32], bool wide) {
    uint8_t* p = row + 2 * static_cast<int64_t>(col);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (wide && col + 16 * i + 16 <= cols) {
            const uint32_t q[8] = {w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3],
                                   w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]};
            st_global_v8(p + 32 * i, q);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (col + 16 * i + 8 * j + 8 <= cols)
                    *reinterpret_cast<uint4*>(p + 32 * i + 16 * j) =
                        make_uint4(w[8 * i + 4 * j], w[8 * i + 4 * j + 1], w[8 * i + 4 * j + 2], w[8 * i + 4 * j + 3]);
        }
    }
}

// 32 fp32 columns of one output row, at once; columns at or past `cols` (a multiple of 8) are left out.
__device__ __forceinline__ void store_fp32(uint8_t* row, int col, int cols, const float (&v)[32], bool wide) {
    uint8_t* p = row + 4 * static_cast<int64_t>(col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (col + 8 * i + 8 > cols) break;
        const uint32_t q[8] = {__float_as_uint(v[8 * i]), __float_as_uint(v[8 * i + 1]), __float_as_uint(v[8 * i + 2]),
                               __float_as_uint(v[8 * i + 3]), __float_as_uint(v[8 * i + 4]), __float_as_uint(v[8 * i + 5]),
                               __float_as_uint(v[8 * i + 6]), __float_as_uint(v[8 * i + 7])};
        if (wide) {
            st_global_v8(p + 32 * i, q);
        } else {
            *reinterpret_cast<uint4*>(p + 32 * i) = make_uint4(q[0], q[1], q[2], q[3]);
            *reinterpret_cast<uint4*>(p + 32 * i + 16) = make_uint4(q[4], q[5], q[6], q[7]);
        }
    }
}

// What a CTA's roles share.
struct Roles {
    const Maps& maps;
    const GemmParams& p;
    const Table& t;
    Control& ctl;
    Waits waits;
    uint8_t* stages;
    uint8_t* boxes;
    uint8_t* residuals;  // a box for each warp
    uint32_t tmem, rank, stage_bytes;  // rank: of the CTA in its pair
    int num_stages, worker, workers;
    bool deep;  // deep_stages()
};

constexpr uint32_t kABytes = kTileRows * kRowBytes;

// One thread: the loads.  kWords: copy_rows() has the row operand.
template <int FORM, int CG, bool kWords>
__device__ __forceinline__ void load_operands(const Roles& x) {
    const GemmParams& p = x.p;
    const Table& t = x.t;
    Control& ctl = x.ctl;
    uint32_t stage = 0, phase = 0;
    uint32_t tail_phase = 0, tail_last = 0;  // per stage: uses of tail_full, mod 2; whether its last use was one
    bool ok = true;
    const uint32_t full0 = CG == 1 ? smem_u32(ctl.full) : cluster_addr(ctl.full, 0);
    uint32_t used = 0;
    for (int tile = x.worker; ok && tile < ctl.tiles; tile += x.workers) {
        const Tile q = decode<FORM, CG>(t, p, ctl, tile);
        const int my_m0 = q.m0 + static_cast<int>(x.rank) * kTileRows;
        const int rows_here = min(kTileRows, q.rows - my_m0);
        const int small_boxes = rows_here > kTileRows / 2 ? 0 : (max(0, rows_here) + kRowBox - 1) / kRowBox;
        uint32_t row_bytes = rows_here > kTileRows / 2 ? kABytes : small_boxes * (kRowBox * kRowBytes);
        if (FORM == kWeightGrad) row_bytes = kABytes;
        else if (kWords) row_bytes = 0;
        const int cols = q.cols / CG;                     // columns that this CTA loads
        const int cb = static_cast<int>(x.rank) * cols;
        const uint32_t bytes = row_bytes + cols * kRowBytes;
        if constexpr (!kWords && FORM != kWeightGrad && FORM != kTransposed) {
            // Every step of the tile loads the same: one or two boxes of rows, one or two of columns, found once.
            const int half = FORM == kGated ? q.cols / 2 : cols;  // gated: the first half of columns are gates, the second their ups
            const int box = half >= kBox ? kBox : kColBox;
            const bool two_rows = small_boxes == 2, two_cols = cols > box;
            auto column = [&](int c) { return q.n0 + (FORM != kGated || c < half ? c : p.cols_dim + c - half); };
            const int at0 = column(cb), at1 = column(cb + box), row = q.row0 + my_m0;
            const CUtensorMap* const rows_map = small_boxes ? &x.maps.a_small : &x.maps.a;
            const CUtensorMap* const cols_map = box == kBox ? &x.maps.b : &x.maps.b_small;
            constexpr int kStep = FORM == kFp8 ? 128 : 64;
            const bool deep = CG == 1 && x.deep;
            const uint32_t step_bytes = kABytes + q.cols / CG * kRowBytes;
            int k0 = q.step0 * kStep;
            auto load = [&](uint8_t* a, uint32_t bar) {
                uint8_t* b = a + kABytes;
                if (rows_here > 0) tma_load_2d<CG>(a, rows_map, k0, row, bar);
                if (two_rows) tma_load_2d<CG>(a + kRowBox * kRowBytes, rows_map, k0, row + kRowBox, bar);
                tma_load_3d<CG>(b, cols_map, k0, at0, q.group, bar);
                if (two_cols) tma_load_3d<CG>(b + box * kRowBytes, cols_map, k0, at1, q.group, bar);
                k0 += kStep;
            };
            for (int s = 0; s < q.steps; ++s) {
                ok = wait_phase(&ctl.empty[stage], phase ^ 1, x.waits);
                if (!ok) break;
                uint8_t* a = x.stages + stage * x.stage_bytes;
                const uint32_t bar = full0 + 8 * stage;
                const bool second = deep && s + 1 < q.steps;
                bar_arrive_expect_tx<CG>(bar, second ? 2 * bytes : bytes);
                load(a, bar);
                if (second) load(a + step_bytes, bar), ++s;
                ++used;
                if (++stage == static_cast<uint32_t>(x.num_stages)) stage = 0, phase ^= 1;
            }
        } else {
            for (int s = 0; s < q.steps; ++s) {
                ok = wait_phase(&ctl.empty[stage], phase ^ 1, x.waits);
                if (!ok) break;
                uint8_t* a = x.stages + stage * x.stage_bytes;
                uint8_t* b = a + kABytes;
                uint32_t bar = full0 + 8 * stage;
                if constexpr (FORM == kWeightGrad) {
                    const bool tail = (s + 1) * 64 > q.rows;
                    if (tail) {
                        bar = smem_u32(&ctl.tail_full[stage]);
                        mbar_arrive_expect_tx(&ctl.tail_full[stage], bytes);
                        tail_phase ^= 1u << stage;
                        tail_last |= 1u << stage;
                    } else {
                        bar_arrive_expect_tx<CG>(bar, bytes);
                        tail_last &= ~(1u << stage);
                    }
                    const int r = q.row0 + s * 64;
                    if (my_m0 + kBox <= p.a_chunked) {
                        tma_load_3d<CG>(a, &x.maps.a, 0, r, my_m0 / 64, bar);
                    } else {
                        tma_load_2d<CG>(a, &x.maps.a_small, my_m0, r, bar);
                        tma_load_2d<CG>(a + 8192, &x.maps.a_small, my_m0 + 64, r, bar);
                    }
                    for (int c = 0; c < cols;) {
                        const int at = q.n0 + cb + c;
                        if (c + kBox <= cols && at + kBox <= p.b_chunked) {
                            tma_load_3d<CG>(b + c * kRowBytes, &x.maps.b, 0, r, at / 64, bar);
                            c += kBox;
                        } else {
                            tma_load_2d<CG>(b + c * kRowBytes, &x.maps.b_small, at, r, bar);
                            c += kColBox;
                        }
                    }
                } else {
                    bar_arrive_expect_tx<CG>(bar, bytes);
                    const int k0 = (q.step0 + s) * (FORM == kFp8 ? 128 : 64);
                    if (small_boxes == 0) {
                        if (!kWords && rows_here > 0) tma_load_2d<CG>(a, &x.maps.a, k0, q.row0 + my_m0, bar);
                    } else if (!kWords) {
                        for (int c = 0; c < small_boxes; ++c)
                            tma_load_2d<CG>(a + c * (kRowBox * kRowBytes), &x.maps.a_small, k0, q.row0 + my_m0 + c * kRowBox, bar);
                    }
                    for (int c = 0; c < cols;) {
                        const int at = q.n0 + cb + c;
                        if (FORM == kTransposed && c + kBox <= cols && at + kBox <= p.b_chunked) {
                            tma_load_4d<CG>(b + c * kRowBytes, &x.maps.b, 0, k0, at / 64, q.group, bar);
                            c += kBox;
                        } else if (FORM == kTransposed) {
                            tma_load_3d<CG>(b + c * kRowBytes, &x.maps.b_small, at, k0, q.group, bar);
                            c += kColBox;
                        } else if (c + kBox <= cols) {
                            tma_load_3d<CG>(b + c * kRowBytes, &x.maps.b, k0, at, q.group, bar);
                            c += kBox;
                        } else {
                            tma_load_3d<CG>(b + c * kRowBytes, &x.maps.b_small, k0, at, q.group, bar);
                            c += kColBox;
                        }
                    }
                }
                ++used;
                if (++stage == static_cast<uint32_t>(x.num_stages)) stage = 0, phase ^= 1;
            }
        }
    }
    // Copies and products in flight end before the memory goes away.  Where all went well the products have read every
    // copy when the last stages are free again, and their arrivals (a pair's at both CTAs) have landed.  Where
    // some warp gave up, each within a limit: the copies that completed a stage, then the products; what a pair has in
    // flight beside that, see the kernel's end.
    for (int i = 0; i < x.num_stages && used > 0; ++i, --used) {
        if (stage == 0) phase ^= 1;
        stage = (stage == 0 ? x.num_stages : stage) - 1;
        if (ok) ok = wait_phase(&ctl.empty[stage], phase, x.waits);
        if (ok) continue;
        const bool tail = (tail_last >> stage) & 1;
        if (x.rank != 0 && !tail) continue;
        uint64_t* bar = tail ? &ctl.tail_full[stage] : &ctl.full[stage];
        const uint32_t parity = tail ? ((tail_phase >> stage) & 1) ^ 1 : phase;
        for (int k = 0; k < (1 << 12) && !mbar_try_wait(bar, parity); ++k) {
        }
    }
    for (int k = 0; k < (1 << 12) && !mbar_try_wait(&ctl.drained, 0); ++k) {
    }
}

// One thread of the pair: the products.
template <int FORM, int CG, bool kWords>
__device__ __forceinline__ void multiply(const Roles& x) {
    constexpr int kSegment = segment_steps(FORM);
    constexpr bool kDeep = CG == 1 && !kWords && (FORM == kForward || has_epilogue(FORM));
    static_assert(kSegment % 2 == 0 || !kDeep, "whole stages a segment");
    const bool deep = kDeep && x.deep;
    const GemmParams& p = x.p;
    const Table& t = x.t;
    Control& ctl = x.ctl;
    uint32_t stage = 0, phase = 0, acc_phase = 0;
    int buf = 0;
    bool ok = true;
    constexpr bool a_mn = FORM == kWeightGrad;
    constexpr bool b_mn = FORM == kWeightGrad || FORM == kTransposed;
    for (int tile = x.worker; ok && tile < ctl.tiles; tile += x.workers) {
        const Tile q = decode<FORM, CG>(t, p, ctl, tile);
        const uint32_t idesc = mma_desc(FORM == kFp8 ? 0 : 1, a_mn, b_mn, kTileRows * CG, q.cols);
        const uint32_t step_bytes = kABytes + q.cols / CG * kRowBytes;
        for (int s = 0; ok && s < q.steps;) {
            const int end = kSegment ? min(q.steps, s + kSegment) : q.steps;  // of an accumulator
            const uint32_t d = x.tmem + buf * kMaxTileCols;
            bool first = true;
            for (; s < end; ++s) {
                // operands first: they are there, and with short segments the accumulator is what is waited for
                if (FORM == kWeightGrad && CG == 2 && q.rows - s * 64 < 64)  // zeroed rows, maybe the peer's
                    ok = wait_phase<true>(&ctl.full[stage], phase, x.waits);
                else
                    ok = wait_phase(&ctl.full[stage], phase, x.waits);
                if (!ok) break;
                if (first) {
                    ok = wait_phase(&ctl.acc_empty[buf], acc_phase ^ 1, x.waits);
                    if (!ok) break;
                }
                tc_fence_after();
                const uint32_t a = smem_u32(x.stages) + stage * x.stage_bytes;
                auto step = [&](uint32_t a) {
                    const uint64_t da = smem_desc(a, a_mn ? 8192 : 16);
                    const uint64_t db = smem_desc(a + kABytes, b_mn ? 8192 : 16);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tc_mma<CG, FORM == kFp8>(d, da + i * (a_mn ? 128 : 2), db + i * (b_mn ? 128 : 2), idesc, !first || i);
                    first = false;
                };
                step(a);
                if (deep && s + 1 < end) step(a + step_bytes), ++s;
                tc_commit<CG>(&ctl.empty[stage]);
                if (++stage == static_cast<uint32_t>(x.num_stages)) stage = 0, phase ^= 1;
            }
            if (!ok) break;
            tc_commit<CG>(&ctl.acc_full[buf]);
            buf ^= 1;
            acc_phase ^= buf == 0;
        }
    }
    // The products already issued still write tensor memory, also where another warp gave up on them: load_operands()
    // waits for this.
    tc_commit<CG>(&ctl.drained);
}

// Two warps: row operands whose rows are not 16 bytes apart (messages of some hidden sizes), in words of four bytes,
// into the place and order in which a tensor-map load puts them.  A warp copies a row's 128 bytes at a time, several
// rows in flight, and waits for them: FP8, 32 experts, n 2048, rows of 2944 bytes 53, 284 and 1500 us at 16, 128 and 1024
// rows an expert, where loads by tensor maps of rows of 3584 take 43, 50 and 200.
template <int FORM>
__device__ __forceinline__ void copy_rows(const Roles& x, int warp) {
    const GemmParams& p = x.p;
    const Table& t = x.t;
    Control& ctl = x.ctl;
    constexpr int kInFlight = FORM == kFp8 ? 8 : 16;  // its registers are fewer
    const int row_bytes = p.contraction * (FORM == kFp8 ? 1 : 2);
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int tile = x.worker; ok && tile < ctl.tiles; tile += x.workers) {
        const Tile q = decode<FORM, 1>(t, p, ctl, tile);
        const int rows = min(kTileRows, q.rows - q.m0);
        for (int s = 0; s < q.steps; ++s) {
            ok = warp_wait(&ctl.empty[stage], phase ^ 1, x.waits);
            if (!ok) break;
            uint8_t* a = x.stages + stage * x.stage_bytes;
            const int at = s * kRowBytes + lane_id() * 4;
            const uint8_t* from = p.a_words + (static_cast<int64_t>(q.row0) + q.m0) * p.a_row_bytes + at;
            for (int r0 = (warp - 2) * kInFlight; r0 < rows; r0 += 2 * kInFlight) {
                uint32_t v[kInFlight];
#pragma unroll
                for (int i = 0; i < kInFlight; ++i)
                    v[i] = r0 + i < rows && at < row_bytes ? *reinterpret_cast<const uint32_t*>(from + (r0 + i) * p.a_row_bytes) : 0;
#pragma unroll
                for (int i = 0; i < kInFlight; ++i) {
                    const int r = r0 + i;  // the 16-byte pieces of a row lie exclusive-or'd with its number
                    *reinterpret_cast<uint32_t*>(a + r * kRowBytes + (((lane_id() >> 2) ^ (r & 7)) << 4) + (lane_id() & 3) * 4) = v[i];
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane_id() == 0) bar_arrive<1>(smem_u32(&ctl.full[stage]));
            if (++stage == static_cast<uint32_t>(x.num_stages)) stage = 0, phase ^= 1;
        }
    }
}

// One warp, weight gradient: the ends of groups.
template <int FORM, int CG>
__device__ __forceinline__ void zero_tails(const Roles& x) {
    const GemmParams& p = x.p;
    const Table& t = x.t;
    Control& ctl = x.ctl;
    // The rows of a group's last, partial block past its end belong to others: zero them in both operands.
    uint32_t stage = 0, tail_phase = 0;  // tail_phase, per stage: uses of tail_full, mod 2
    bool ok = true;
    for (int tile = x.worker; ok && tile < ctl.tiles; tile += x.workers) {
        const Tile q = decode<FORM, CG>(t, p, ctl, tile);
        const int whole = q.rows / 64, valid = q.rows % 64;
        stage = (stage + whole) % x.num_stages;
        if (valid == 0) continue;
        ok = warp_wait(&ctl.tail_full[stage], (tail_phase >> stage) & 1, x.waits);
        if (!ok) break;  // a copy may still be on its way there
        tail_phase ^= 1u << stage;
        uint8_t* a = x.stages + stage * x.stage_bytes;
        const int chunks = (kTileRows + q.cols / CG) / 64;
        const int pieces = (64 - valid) * 8;
        for (int c = 0; c < chunks; ++c) {
            uint4* z = reinterpret_cast<uint4*>(a + c * 8192 + valid * 128);
            for (int i = lane_id(); i < pieces; i += kWarpSize) z[i] = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        __syncwarp();
        if (lane_id() == 0)
            bar_arrive_written<CG>(CG == 1 ? smem_u32(&ctl.full[stage]) : cluster_addr(&ctl.full[stage], 0));
        stage = (stage + 1) % x.num_stages;
    }
}

// 32 columns of a lane's row, rounded to bf16, into the first or second half of its warp's box of 32 rows by 64
// columns; 16-byte pieces lie exclusive-or'd with the row's number.
__device__ __forceinline__ void box_columns(uint32_t box, int second, const float (&v)[32]) {
    const uint32_t row = box + lane_id() * kRowBytes;
    const uint32_t turn = lane_id() & 7;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
        st_shared_v4(row + (((second * 4 + j) ^ turn) << 4), w);
    }
}

// 32 fp32 columns of a lane's row into its warp's box of 32 rows by 32 columns.
__device__ __forceinline__ void box_columns_fp32(uint32_t box, const float (&v)[32]) {
    const uint32_t row = box + lane_id() * kRowBytes;
    const uint32_t turn = lane_id() & 7;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w[4] = {__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                               __float_as_uint(v[4 * j + 3])};
        st_shared_v4(row + ((j ^ turn) << 4), w);
    }
}

// 32 columns of a warp's rows, from column `c` of its part of the tile.  kStaged: through the warp's boxes in shared
// memory, 128 bytes of columns at a time (the map leaves out what lies past the last column, and in the weight gradient
// past the last row).  Otherwise by stores of each lane.
template <int FORM, bool kStaged>
__device__ __forceinline__ void put_columns(const Roles& x, uint32_t box, const Place& at, int c, const float (&v)[32]) {
    const GemmParams& p = x.p;
    const int col = at.col + c;
    if constexpr (FORM == kWeightGrad && kStaged) {
        if (at.rows == 0 || col >= p.cols_dim) return;
        if (lane_id() == 0) bulk_wait_read<0>();
        __syncwarp();
        box_columns_fp32(box, v);
        fence_async_smem();
        __syncwarp();
        if (lane_id() == 0) {
            if (p.accumulate) tma_add_3d(&x.maps.out, box, col, at.row, at.group);
            else tma_store_3d(&x.maps.out, box, col, at.row, at.group);
            bulk_commit();
        }
    } else if constexpr (kStaged) {
        constexpr int kBoxes = out_boxes(FORM);
        const int second = (c >> 5) & 1;
        const int first_col = col - 32 * second;
        box += (c >> 6 & (kBoxes - 1)) * kOutBox;
        if (first_col < p.cols_dim) {
            if (!second) {  // the last copy out of this box has read it: boxes take turns
                if (lane_id() == 0) bulk_wait_read<kBoxes - 1>();
                __syncwarp();
            }
            box_columns(box, second, v);
        }
        if (!second) return;
        fence_async_smem();
        __syncwarp();
        if (lane_id() == 0) {
            if (first_col < p.cols_dim) tma_store_2d(&x.maps.out, box, first_col, at.row);
            bulk_commit();                                   // empty past the last column: a turn all the same
            if (kBoxes == 2 && at.cols == 64) bulk_commit();  // the second box's
        }
    } else if (lane_id() < at.rows && col < p.cols_dim) {
        const int64_t row = (FORM == kWeightGrad ? static_cast<int64_t>(at.group) * p.rows_dim : 0) + at.row + lane_id();
        uint8_t* out = static_cast<uint8_t*>(p.out) + row * p.out_row_bytes;
        if (FORM == kActivatedFp32) store_fp32(out, col, p.cols_dim, v, p.wide_stores != 0);
        else store_bf16(out, col, p.cols_dim, v, p.wide_stores != 0);
    }
}

// A warp's box of the residual: 32 rows by 64 columns.  By tensor map, not by the lanes: of 227 KB of shared memory the L1
// cache keeps nothing, and loads of 32 rows at once wait for its few lines (8187 rows, 7168 x 2048: 245 us, 123 without a
// residual).  One box, since two leave four stages of a pair's operands instead of six (161 us).
constexpr uint32_t kResidualBytes = kEpilogueWarps * kOutBox;

// What a warp asks for of its part of a tile before the tile's sums are there: the bias, lane l columns 4 l to 4 l + 3, and
// the residual.
template <int FORM>
struct Ahead {
    float4 bias, up_bias;
    uint8_t* box;
    uint64_t* arrived;
    uint32_t phase;
    bool asked;

    __device__ __forceinline__ Ahead(const Roles& x, int w)
        : box(x.residuals + w * kOutBox), arrived(&x.ctl.tail_full[w]), phase(0), asked(false) {}
    __device__ __forceinline__ void load_bias(const GemmParams& p, const Place& at) {
        bias = up_bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p.bias == nullptr || 4 * lane_id() >= at.cols || at.col + 4 * lane_id() >= p.cols_dim) return;
        const float* from = p.bias + static_cast<int64_t>(at.group) * (FORM == kGated ? 2 : 1) * p.cols_dim + at.col + 4 * lane_id();
        bias = __ldg(reinterpret_cast<const float4*>(from));
        if (FORM == kGated) up_bias = __ldg(reinterpret_cast<const float4*>(from + p.cols_dim));
    }
    // 64 columns from column c of the warp's part, after the warp has read what is there.
    __device__ __forceinline__ void ask_residual(const Roles& x, const Place& at, int c) {
        asked = x.p.residual != nullptr && at.rows > 0 && c < at.cols && at.col + c < x.p.cols_dim;
        if (!asked) return;
        __syncwarp();
        if (lane_id() == 0) {
            mbar_arrive_expect_tx(arrived, kOutBox);
            tma_load_2d<1>(box, &x.maps.residual, at.col + c, at.row, smem_u32(arrived));
        }
    }
    __device__ __forceinline__ bool wait_residual(const Waits& waits) {
        if (!asked) return true;
        if (!warp_wait(arrived, phase, waits)) return false;
        asked = false;
        phase ^= 1;
        return true;
    }
    // Of a wait that was given up: the copy ends before the memory goes away.
    __device__ __forceinline__ void leave() {
        for (int k = 0; asked && k < (1 << 8) && !mbar_try_wait(arrived, phase); ++k) {
        }
    }
};

// v += 32 columns of the bias from column `c` of the warp's part, which the lanes hold.
__device__ __forceinline__ void add_bias(const float4& bias, int c, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int from = c / 4 + i;
        v[4 * i] += __shfl_sync(kFullMask, bias.x, from);
        v[4 * i + 1] += __shfl_sync(kFullMask, bias.y, from);
        v[4 * i + 2] += __shfl_sync(kFullMask, bias.z, from);
        v[4 * i + 3] += __shfl_sync(kFullMask, bias.w, from);
    }
}

// After a warp's sums of a part of a tile are written: whether they are the last of the tile's, and all may be read.  Each
// warp of a CTA meets its like in the others, so that the CTA does not wait.
__device__ __forceinline__ bool last_part(const GemmParams& p, int meeting, int parts) {
    __syncwarp();
    int before = 0;
    if (lane_id() == 0) {
        before = arrive_at(p.tickets + meeting);
        if (before == parts - 1) p.tickets[meeting] = 0;  // for the next call
    }
    __syncwarp();
    return __shfl_sync(kFullMask, before, 0) == parts - 1;
}

// 32 columns from c of a warp's sums, the parts in their order, two on their way at a time.
__device__ __forceinline__ void sum_parts(const GemmParams& p, int meeting, int parts, int c, float (&v)[32]) {
    const float* from = p.parts + static_cast<int64_t>(meeting) * parts * kPartFloats + c * kWarpSize + lane_id();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __ldcg(from + i * kWarpSize);
    for (int k = 1; k < parts; k += 2) {
        float one[32], two[32];
        from += kPartFloats;
#pragma unroll
        for (int i = 0; i < 32; ++i) one[i] = __ldcg(from + i * kWarpSize);
        const bool more = k + 1 < parts;
        if (more) from += kPartFloats;
#pragma unroll
        for (int i = 0; i < 32; ++i) two[i] = more ? __ldcg(from + i * kWarpSize) : 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = v[i] + one[i] + two[i];
    }
}

template <int ACT>
__device__ __forceinline__ void activate_columns(float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float2 a = activate(ACT, make_float2(v[i], v[i + 1]));
        v[i] = a.x, v[i + 1] = a.y;
    }
}

// The epilogue of 32 output columns of a lane's row, from column `c` of its warp's part of the tile: v holds the sums
// (gated: of the gates, and `up` of the ups) and gets what is written.  False: the wait for the residual was given up.
template <int FORM>
__device__ __forceinline__ bool finish_columns(const Roles& x, const Place& at, int c, Ahead<FORM>& ahead, float (&v)[32], float (&up)[32]) {
    const GemmParams& p = x.p;
    const int col = at.col + c;
    if (col >= p.cols_dim) return true;
    const int64_t row = static_cast<int64_t>(at.row) + lane_id();
    const bool in = lane_id() < at.rows;
    if (p.bias) {
        add_bias(ahead.bias, c, v);
        if (FORM == kGated) add_bias(ahead.up_bias, c, up);
    }
    if (p.pre && in) {
        uint8_t* pre = p.pre + row * p.pre_row_bytes;
        store_bf16(pre, col, p.cols_dim, v, p.pre_wide != 0);
        if (FORM == kGated) store_bf16(pre + 2 * static_cast<int64_t>(p.cols_dim), col, p.cols_dim, up, p.pre_wide != 0);
    }
    switch (p.act) {  // the same for all: a loop each, not a choice for each value
        case EP_ACT_RELU: activate_columns<EP_ACT_RELU>(v); break;
        case EP_ACT_SILU: activate_columns<EP_ACT_SILU>(v); break;
        case EP_ACT_GELU: activate_columns<EP_ACT_GELU>(v); break;
        default: break;
    }
    if (FORM == kGated) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= up[i];
    }
    if (p.row_weights) {
        const float w = in ? p.row_weights[row] : 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= w;
    }
    if (p.residual) {
        if (!ahead.wait_residual(x.waits)) return false;
        const uint8_t* from = ahead.box + lane_id() * kRowBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 16-byte pieces lie exclusive-or'd with the row's number
            float r[8];
            unpack8(*reinterpret_cast<const int4*>(from + ((((c >> 5 & 1) * 4 + i) ^ (lane_id() & 7)) << 4)), r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * i + j] += r[j];
        }
        if (c & 32) ahead.ask_residual(x, at, c + 32);
    }
    return true;
}

// Whether a warp's part of a tile leaves through its boxes: not the ends of groups, nor tiles of 64 columns.  Asked once a
// tile (64 experts of 2048 rows, 7168 x 2048 in FP8: 1692 us asked for every 32 columns, 1679 so).
template <int FORM>
__device__ __forceinline__ bool in_boxes(const GemmParams& p, const Place& at) {
    return p.staged && (FORM == kWeightGrad || (at.cols >= 64 && at.rows == 32));
}

// A warp's sums, 128 columns a lane at most, to their place.
template <int FORM, bool kStaged>
__device__ __forceinline__ void put_sums(const Roles& x, uint32_t box, const Place& at, const uint64_t (&acc)[2][32]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (32 * c >= at.cols) break;
        float v[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint64_t pair = acc[c / 2][c % 2 * 16 + i];
            v[2 * i] = __uint_as_float(static_cast<uint32_t>(pair));
            v[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(pair >> 32));
        }
        put_columns<FORM, kStaged>(x, box, at, 32 * c, v);
    }
}

// The same after their epilogue, by stores of each lane; meeting >= 0: of a tile's parts, from there.
template <int FORM>
__device__ __forceinline__ bool put_finished(const Roles& x, const Place& at, Ahead<FORM>& ahead, const uint64_t (&acc)[2][32], int meeting) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (32 * c >= at.cols) break;
        float v[32];
        if (meeting >= 0) {
            sum_parts(x.p, meeting, x.ctl.parts, 32 * c, v);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint64_t pair = acc[c / 2][c % 2 * 16 + i];
                v[2 * i] = __uint_as_float(static_cast<uint32_t>(pair));
                v[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(pair >> 32));
            }
        }
        if (!finish_columns<FORM>(x, at, 32 * c, ahead, v, v)) return false;
        put_columns<FORM, false>(x, 0, at, 32 * c, v);
    }
    return true;
}

// Eight warps: accumulators to the output.
template <int FORM, int CG>
__device__ __forceinline__ void store_tiles(const Roles& x, int warp) {
    constexpr int kSegment = segment_steps(FORM);
    const GemmParams& p = x.p;
    const Table& t = x.t;
    Control& ctl = x.ctl;
    const int w = warp - 4;
    const int quarter = warp & 3;               // the 32 lanes of tensor memory that this warp may read
    const int half = w >> 2;                    // which half of the tile's columns
    const uint32_t lane_base = x.tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t acc_empty0 = CG == 1 ? smem_u32(ctl.acc_empty) : cluster_addr(ctl.acc_empty, 0);
    const uint32_t box = smem_u32(x.boxes) + w * (out_boxes(FORM) * kOutBox);
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    Ahead<FORM> ahead(x, w);
    const bool cut = has_epilogue(FORM) && ctl.parts > 1;  // then the tickets are taken also after a wait was given up
    for (int tile = x.worker; (ok || cut) && tile < ctl.tiles; tile += x.workers) {
        const Tile q = decode<FORM, CG>(t, p, ctl, tile);
        const int meeting = (q.tile * CG + static_cast<int>(x.rank)) * kEpilogueWarps + w;  // of a tile's parts
        float* const part = cut ? p.parts + (static_cast<int64_t>(meeting) * ctl.parts + (tile - q.tile * ctl.parts)) * kPartFloats + lane_id() : nullptr;
        if (FORM == kWeightGrad && p.accumulate && q.steps == 0) continue;  // nothing to add
        const int cols_half = out_cols<FORM>(q.cols) / 2;
        const int in_group = q.m0 + static_cast<int>(x.rank) * kTileRows + quarter * 32;
        const int rows = min(32, max(0, (FORM == kWeightGrad ? p.rows_dim : q.rows) - in_group));
        const Place at = {(FORM == kWeightGrad ? 0 : q.row0) + in_group, q.n0 + half * cols_half, q.group,
                          static_cast<short>(rows), static_cast<short>(cols_half)};
        // Whether this warp has nothing of the tile, in any of its parts: with up to 32 rows three of four warps, which then neither
        // write nor meet (16 rows, 1024 x 7168: 10.8 to 10.2 us, gated 15.4 to 14.2; without parts no change).
        const bool nothing = has_epilogue(FORM) && (rows == 0 || at.col >= p.cols_dim);
        if (!ok) {
            if (!nothing) last_part(p, meeting, ctl.parts);
            continue;
        }
        if constexpr (has_epilogue(FORM)) {
            if (!nothing) ahead.load_bias(p, at);
            if (!cut) ahead.ask_residual(x, at, 0);
        }
        if constexpr (kSegment == 0) {
            ok = warp_wait(&ctl.acc_full[buf], acc_phase, x.waits);
            if (!ok) {
                if (!cut) break;
                if (!nothing) last_part(p, meeting, ctl.parts);
                continue;
            }
            tc_fence_after();
            if (nothing) {
                tc_fence_before();
                __syncwarp();
                if (lane_id() == 0) bar_arrive<CG>(acc_empty0 + 8 * buf);
                buf ^= 1;
                acc_phase ^= buf == 0;
                continue;
            }
            const bool staged = in_boxes<FORM>(p, at);
            bool mine = true;  // this warp's to finish
            if (cut) {
                for (int c = 0; c < (FORM == kGated ? 2 : 1) * cols_half; c += 32) {
                    uint32_t u[32];
                    __syncwarp();
                    const int at_up = FORM == kGated && c >= cols_half ? q.cols / 2 - cols_half : 0;
                    tc_ld32(lane_base + buf * kMaxTileCols + half * cols_half + c + at_up, u);
                    tc_wait_ld(u);
#pragma unroll
                    for (int i = 0; i < 32; ++i) part[(c + i) * kWarpSize] = __uint_as_float(u[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane_id() == 0) bar_arrive<CG>(acc_empty0 + 8 * buf);
                mine = last_part(p, meeting, ctl.parts);
                if constexpr (has_epilogue(FORM))
                    if (mine) ahead.ask_residual(x, at, 0);
            }
            for (int c = 0; mine && c < cols_half; c += 32) {
                float v[32], up[32];  // up: gated
                if (cut) {
                    sum_parts(p, meeting, ctl.parts, c, v);
                    if (FORM == kGated) sum_parts(p, meeting, ctl.parts, cols_half + c, up);
                } else {
                    uint32_t u[32];
                    __syncwarp();
                    const uint32_t from = lane_base + buf * kMaxTileCols + half * cols_half + c;
                    tc_ld32(from, u);
                    if constexpr (FORM == kGated) {
                        uint32_t u2[32];
                        tc_ld32(from + q.cols / 2, u2);
                        tc_wait_ld(u2);
#pragma unroll
                        for (int i = 0; i < 32; ++i) up[i] = __uint_as_float(u2[i]);
                    }
                    tc_wait_ld(u);
                    if (c + 32 >= cols_half) {  // read out: the accumulator is free before the last stores
                        tc_fence_before();
                        __syncwarp();
                        if (lane_id() == 0) bar_arrive<CG>(acc_empty0 + 8 * buf);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
                }
                if constexpr (has_epilogue(FORM)) {
                    ok = ok && finish_columns<FORM>(x, at, c, ahead, v, up);
                    if (!ok) continue;  // the accumulator is freed all the same
                }
                if (staged) put_columns<FORM, true>(x, box, at, c, v);
                else put_columns<FORM, false>(x, box, at, c, v);
            }
            buf ^= 1;
            acc_phase ^= buf == 0;
        } else {
            // The sums of a segment arrive in an accumulator of their own and are added up here, 128 columns a
            // thread at most; in FP8 a segment is a block of 128 with its own scales.  Meanwhile the tile's place
            // lies in shared memory: there are no registers for it.
            uint64_t acc[2][32];  // pairs of fp32
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[c][i] = 0;
            if (lane_id() == 0) ctl.at[w] = at;
            const int segments = (q.steps + kSegment - 1) / kSegment;
            // A block's scales are loaded a block before they are used, and only then looked at: a
            // multiplication next to the loads would wait for them.  All of it comes before the wait for the block's
            // products, and without a branch (the last block loads its own scales again): 8 experts of 2048 rows,
            // 4096 x 7168, 381 us with a branch after the wait, 369 without it, 362 so.
            const uint8_t* xs = nullptr;
            const float* ws = nullptr;
            uint32_t x_next = 0;
            float w_next = 0.0f;
            if constexpr (FORM == kFp8) {
                xs = p.x_scales + (static_cast<int64_t>(q.row0) + min(in_group + lane_id(), q.rows - 1)) * p.x_scale_row_bytes;
                const int nb = min(at.col, p.cols_dim - 1) >> 7;
                ws = p.w_scales + (static_cast<int64_t>(q.group) * ((p.cols_dim + 127) >> 7) + nb) * q.steps;
                x_next = raw_scale(xs, 0, p.scales_ue8m0);
                w_next = ws[0];
            }
#pragma unroll 1
            for (int left = segments; left > 0; --left) {
                float f = 1.0f;
                if constexpr (FORM == kFp8) {
                    f = scale_value(x_next, p.scales_ue8m0) * w_next;
                    const int on = left > 1;
                    xs += p.scales_ue8m0 ? on : 4 * on;
                    ws += on;
                    x_next = raw_scale(xs, 0, p.scales_ue8m0);
                    w_next = *ws;
                }
                ok = warp_wait(&ctl.acc_full[buf], acc_phase, x.waits);
                if (!ok) break;
                tc_fence_after();
                const uint32_t from = lane_base + buf * kMaxTileCols + half * cols_half;
                uint32_t u[64];
                tc_ld64(from, u);
                const uint64_t scale = pack_f32x2(__float_as_uint(f), __float_as_uint(f));
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    tc_wait_ld(u);
                    if (c == 1 || cols_half <= 64) {  // all read: the accumulator is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane_id() == 0) bar_arrive<CG>(acc_empty0 + 8 * buf);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) fma_f32x2(acc[c][i], pack_f32x2(u[2 * i], u[2 * i + 1]), scale);
                    if (cols_half <= 64) break;
                    if (c == 0) tc_ld64(from + 64, u);
                }
                buf ^= 1;
                acc_phase ^= buf == 0;
            }
            __syncwarp();
            if (!ok) {
                if (!cut) break;
                if (!nothing) last_part(p, meeting, ctl.parts);
                continue;
            }
            if (nothing) continue;
            if (cut) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (32 * c >= cols_half) break;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t two = acc[c / 2][c % 2 * 16 + i];
                        part[(32 * c + 2 * i) * kWarpSize] = __uint_as_float(static_cast<uint32_t>(two));
                        part[(32 * c + 2 * i + 1) * kWarpSize] = __uint_as_float(static_cast<uint32_t>(two >> 32));
                    }
                }
                if (!last_part(p, meeting, ctl.parts)) continue;
                if constexpr (has_epilogue(FORM)) ahead.ask_residual(x, at, 0);
            }
            const Place to = read_place(&ctl.at[w]);
            if constexpr (has_epilogue(FORM)) {
                ok = put_finished<FORM>(x, to, ahead, acc, cut ? meeting : -1);
            } else if (in_boxes<FORM>(p, to)) put_sums<FORM, true>(x, box, to, acc);
            else put_sums<FORM, false>(x, box, to, acc);
            __syncwarp();  // the place has been read
        }
    }
    if constexpr (has_epilogue(FORM)) ahead.leave();
    if (lane_id() == 0) bulk_wait_all();
    __syncwarp();
}

// kWords (single CTAs only): rows in words of four bytes, by two more warps.  A kernel of its own: its code in the
// others took registers from the FP8 form's sums (334 to 414 us on messages of 64 experts).
template <int FORM, int CG, bool kWords = false>
__global__ void __launch_bounds__(kGemmThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ Maps maps, const GemmParams p) {
    extern __shared__ uint8_t raw[];
    __shared__ Control ctl;
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Table t;
    t.before = reinterpret_cast<int32_t*>(smem);
    t.count = t.before + p.groups.groups + 1;
    t.begin = t.count + p.groups.groups;
    const uint32_t table_end = (4u * (3u * p.groups.groups + 1u) + 1023u) & ~1023u;
    uint8_t* const boxes = smem + table_end;
    uint32_t out_bytes = p.staged ? kEpilogueWarps * out_boxes(FORM) * kOutBox : 0;
    uint8_t* const residuals = boxes + out_bytes;
    if (has_epilogue(FORM) && p.residual) out_bytes += kResidualBytes;
    uint8_t* const stages = boxes + out_bytes;

    const int warp = threadIdx.x / kWarpSize;
    const uint32_t rank = CG == 1 ? 0 : cluster_rank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&ctl.full[i], CG + (kWords ? 2 : 0));
            mbar_init(&ctl.empty[i], 1);
            mbar_init(&ctl.tail_full[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.acc_full[i], 1);
            mbar_init(&ctl.acc_empty[i], kEpilogueWarps * CG);
        }
        mbar_init(&ctl.drained, 1);
        ctl.abort_flag = 0;
        fence_barrier_init();
        prefetch_map(&maps.a);
        prefetch_map(&maps.b);
    }
    if (warp == 1) tmem_alloc<CG>(&ctl.tmem, 512);
    pdl_enter();
    build_table<FORM, CG>(t, p, ctl);
    tc_fence_before();
    if constexpr (CG == 2) cluster_barrier();
    else __syncthreads();
    tc_fence_after();

    const bool deep = deep_stages<FORM, CG, kWords>(ctl.tile_cols);
    const uint32_t stage_bytes = (deep ? 2 : 1) * (kABytes + ctl.tile_cols / CG * kRowBytes);
    const Roles x = {maps, p, t, ctl, {&ctl.abort_flag, p.status, p.wait_limit_ns}, stages, boxes, residuals, ctl.tmem, rank, stage_bytes,
                     min(kMaxStages, static_cast<int>((kMaxSmem - 1024u - table_end - out_bytes) / stage_bytes)),
                     static_cast<int>(blockIdx.x / CG), static_cast<int>(gridDim.x / CG), deep};
    // Forms with segments hold 128 sums a thread in their eight epilogue warps: registers move there from the
    // others (72 + 2 * 216 = 3 * 168, what the block was launched with).
    constexpr bool kSums = segment_steps(FORM) != 0;
    if (warp < 4) {
        if constexpr (kSums) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0) {
            if (elect_one()) load_operands<FORM, CG, kWords>(x);
        } else if (warp == 1) {
            if (rank == 0 && elect_one()) multiply<FORM, CG, kWords>(x);
        } else if (FORM == kWeightGrad && warp == 2) {
            zero_tails<FORM, CG>(x);
        } else if (kWords) {
            copy_rows<FORM>(x, warp);
        }
    } else {
        if constexpr (kSums) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        store_tiles<FORM, CG>(x, warp);
    }
    __syncwarp();
    tc_fence_before();
    if constexpr (CG == 2) {
        cluster_barrier();
        // Given up (both CTAs have the flag): a stage that only one of the two has loaded completes no barrier, so its copy
        // is given a hundred times what a copy takes, instead of being waited for.
        if (x.waits.abort_flag[0]) {
            if (threadIdx.x == 0)
                for (const uint64_t begin = global_ns(); global_ns() - begin < 1000000;) __nanosleep(1000);
            __syncwarp();
            cluster_barrier();
        }
    } else {
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 1) tmem_dealloc<CG>(x.tmem, 512);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Rows [rows][inner] with a row stride.
Operand row_operand(const void* base, bool fp8, uint64_t inner, uint64_t rows, uint64_t row_bytes, uint32_t box_rows) {
    return {base, fp8 ? Element::kFp8 : Element::kBf16, 2, {inner, rows, 1, 1}, {row_bytes, 0, 0}, {fp8 ? 128u : 64u, box_rows, 1, 1}};
}

// The same rows read across, 64 columns by 64 rows; `chunks` of 64 columns in one load.  With more than one, a chunk
// is an index of its own and the map ends at the last whole one (chunked_columns): a partial one would reach into
// the next row, and past the last row's end.
int chunked_columns(int inner) { return inner >= kBox ? inner / 64 * 64 : 0; }

Operand across_operand(const void* base, uint64_t inner, uint64_t rows, uint64_t row_bytes, uint32_t chunks) {
    if (chunks == 1) return row_operand(base, false, inner, rows, row_bytes, 64);
    return {base, Element::kBf16, 3, {64, rows, inner / 64, 1}, {row_bytes, 128, 0}, {64, 64, chunks, 1}};
}

// Weights [groups][rows][inner], contiguous.
Operand weight_operand(const void* base, bool fp8, uint64_t inner, uint64_t rows, uint64_t groups, uint32_t box_rows) {
    const uint64_t row = inner * (fp8 ? 1 : 2);
    return {base, fp8 ? Element::kFp8 : Element::kBf16, 3, {inner, rows, groups, 1}, {row, row * rows, 0}, {fp8 ? 128u : 64u, box_rows, 1, 1}};
}

Operand weight_across_operand(const void* base, uint64_t inner, uint64_t rows, uint64_t groups, uint32_t chunks) {
    if (chunks == 1) return weight_operand(base, false, inner, rows, groups, 64);
    const uint64_t row = inner * 2;
    return {base, Element::kBf16, 4, {64, rows, inner / 64, groups}, {row, 128, row * rows}, {64, 64, chunks, 1}};
}

// Whether results go out through shared memory: tensor-map stores of 4 KB take a warp less time than its lanes' stores of
// 32 bytes, or of 16 where rows are not 32 bytes aligned, but cost operand stages.
//   - bf16: the lanes' stores run under the next tile's products and only short tiles wait for them.  Without and with, 64
//     experts of 1024 rows, k 256, 512, 1024, 2048: 172 and 138 us, 224 and 215, 356 and 366, 658 and 674 for n = 4096;
//     320 and 163, 295 and 254, 408 and 387, 702 and 700 for n = 4104.
//   - FP8: its sums always wait for them.  k 512, 2048, 7168, n = 4096: 32 experts of 2048 rows (pairs) 258 and 213, 553 and
//     495, 1519 and 1475; 64 of 700 (single CTAs) 183 and 153, 412 and 387, 1143 and 1156; 64 of 128 52 and 45, 114 and 114,
//     329 and 342 (k 4096: 202 and 207, 727 and 707 of 700).
//   - Weight gradient in fp32: always.  Without and with, 32 experts, 2048 x 2048, 16, 512, 1024, 1536, 2048 rows: 134 and 89
//     us, 136 and 135, 200 and 197, 284 and 265, 351 and 330; of 2048 rows, 2048 x 7168, 1179 and 1125; 16 experts of 2048
//     rows, 1680 x 3480, 300 and 283 (768 rows an accumulator).  Added to what is there the lanes would wait for it to
//     arrive (the copy adds in the L2 cache, each element once): 16 rows 316 and 215, 2048 rows 498 and 368 (768).
template <int FORM>
bool staged_pays(bool pairs, const GemmParams& p, int64_t rows_each) {
    if (FORM == kWeightGrad) return p.out_fp32;
    if (rows_each < kRowBox || p.out_fp32) return false;  // no whole block; fp32 rows (activated form) go out by lanes
    if (FORM != kFp8) return !p.wide_stores || p.contraction <= 512;
    return pairs || p.contraction <= (rows_each > 2 * kTileRows ? 4096 : 2048);
}

// Whether the weight gradient runs on pairs of CTAs: its tiles are known here, and it is the side whose waves take less.
// A stage takes 2 cycles a column of products or 3 for two rows of operands that a CTA loads, whichever is longer.
// Measured, pairs against single CTAs where the model prefers these, 1500 and 256 rows an expert: 64 experts of 344 x 4096
// 311 and 293 us, 101 and 87; 8 of 560 x 2448 49.0 and 45.2, 20.0 and 17.8; where it prefers pairs: 8 of 2048 x 2048 76 and
// 89, 31 and 32; 16 of 392 x 2048 54 and 59, 21 and 22.  Groups of more than 1536 rows always on pairs: their operands no
// longer wait in the L2 cache for the next tile (8 experts of 10449 rows, 560 x 2448: 250 and 305).
bool wgrad_on_pairs(const ep_handle* h, const GemmParams& p) {
    if (p.rows_dim <= kTileRows) return false;  // one of the two would idle
    if (p.groups.num_rows > INT64_C(1536) * p.groups.groups) return h->plan.gemm_pairs > 0;
    int64_t best[2];
    for (int ctas = 1; ctas <= 2; ++ctas) {
        const int64_t workers = ctas == 2 ? h->plan.gemm_pairs : h->plan.num_sms;
        if (workers == 0) return false;
        best[ctas - 1] = INT64_MAX;
        for (int cols = kMaxTileCols; cols >= kColBox * ctas; cols >>= 1) {
            const int64_t rows = kTileRows * ctas;
            const int64_t tiles = p.groups.groups * ((p.rows_dim + rows - 1) / rows) * ((p.cols_dim + cols - 1) / cols);
            const int64_t stage = 4 * cols > 3 * (kTileRows + cols / ctas) ? 4 * cols : 3 * (kTileRows + cols / ctas);
            const int64_t cost = (tiles + workers - 1) / workers * stage;
            if (cost < best[ctas - 1]) best[ctas - 1] = cost;
        }
    }
    return best[1] <= best[0];
}

// Forms that read rows in words of four bytes.
constexpr bool has_words(int form) { return form != kWeightGrad && !has_epilogue(form); }

// Whether a product with an epilogue has a tile for every pair of CTAs.  With fewer, as for a router's few columns, single
// CTAs take twice as many narrower ones.
template <int FORM>
bool fills_pairs(const GemmParams& p, int64_t rows_each, int pairs) {
    constexpr int64_t kRows = 2 * kTileRows, kCols = FORM == kGated ? kColBox : 2 * kColBox;
    return p.groups.groups * ((rows_each + kRows - 1) / kRows) * ((p.cols_dim + kCols - 1) / kCols) >= pairs;
}

template <int FORM>
cudaError_t plan_form(LaunchPlan* plan) {
    cudaError_t err = cudaFuncSetAttribute(grouped_gemm_kernel<FORM, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(grouped_gemm_kernel<FORM, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (err == cudaSuccess && has_words(FORM))
        err = cudaFuncSetAttribute(grouped_gemm_kernel<FORM, 1, has_words(FORM)>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   kMaxSmem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan->num_sms / 2 * 2);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int pairs = 0;
    if (plan->num_sms >= 2) err = cudaOccupancyMaxActiveClusters(&pairs, grouped_gemm_kernel<FORM, 2>, &cfg);
    if (err != cudaSuccess) return err;
    int* const least = has_epilogue(FORM) ? &plan->act_pairs : &plan->gemm_pairs;
    if (pairs < *least) *least = pairs;
    return cudaSuccess;
}

// The pairs of CTAs that are resident at once.
cudaError_t plan_gemm(LaunchPlan* plan) {
    plan->gemm_pairs = plan->num_sms / 2;
    cudaError_t err = plan_form<kForward>(plan);
    if (err == cudaSuccess) err = plan_form<kTransposed>(plan);
    if (err == cudaSuccess) err = plan_form<kWeightGrad>(plan);
    if (err == cudaSuccess) err = plan_form<kFp8>(plan);
    return err;
}

// The same for the forms with an epilogue, whose kernels the others' callers do not load.
cudaError_t plan_act(LaunchPlan* plan) {
    plan->act_pairs = plan->num_sms / 2;
    cudaError_t err = plan_form<kActivated>(plan);
    if (err == cudaSuccess) err = plan_form<kActivatedFp32>(plan);
    return err == cudaSuccess ? plan_form<kGated>(plan) : err;
}

template <int FORM>
ep_status launch(ep_handle* h, const Operand& a, const Operand& a_small, const Operand& b, const Operand& b_small,
                 GemmParams p, int64_t rows_each, cudaStream_t stream) {
    DeviceGuard guard(h->device);
    const ep_status planned = has_epilogue(FORM) ? plan_once(&h->plan.act_ready, [h] { return plan_act(&h->plan); })
                                                 : plan_once(&h->plan.gemm_ready, [h] { return plan_gemm(&h->plan); });
    if (planned != EP_OK) return planned;
    const int most_pairs = has_epilogue(FORM) ? h->plan.act_pairs : h->plan.gemm_pairs;
    Maps m;
    const bool pairs = FORM == kWeightGrad ? wgrad_on_pairs(h, p)
                                           : !p.a_words && rows_each >= (FORM == kFp8 ? kPairRowsFp8 : kTileRows + 1) &&
                                                 most_pairs > 0 && (!has_epilogue(FORM) || (!p.parts && fills_pairs<FORM>(p, rows_each, most_pairs)));
    // A tile's stages wait for their operands, and a tile is worth the rows that a CTA loads beside its columns: a pair's
    // 128 beside half of the columns (weight gradient of 8 experts, 560 x 2448, 83592 rows: 401 us with 32 columns'
    // worth, 257 with 128, 246 with 256), a single CTA's as many as a group's tiles have, at least one load's (FP8, 64
    // experts, 1560 x 7168, against always 32: 256 rows an expert 311 and 233 us, 512 550 and 396, 100 163 and 147; always
    // 128: decode steps up to 8 % slower).
    const int64_t row_tiles = (rows_each + kTileRows - 1) / kTileRows;
    p.tile_overhead = pairs                 ? 2 * kTileRows
                      : FORM == kWeightGrad ? kTileRows
                                            : static_cast<int32_t>(rows_each < kRowBox ? kRowBox : rows_each / row_tiles);
    p.staged = staged_pays<FORM>(pairs, p, rows_each);
    ep_status st = encode(&m.b, b);
    if (st == EP_OK) st = encode(&m.b_small, b_small);
    m.out = m.b;  // not used
    if (st == EP_OK && p.staged) {
        const uint64_t cols = p.cols_dim, row = p.out_row_bytes;
        if (FORM == kWeightGrad)
            st = encode(&m.out, {p.out, Element::kFp32, 3, {cols, static_cast<uint64_t>(p.rows_dim), static_cast<uint64_t>(p.groups.groups), 1},
                                 {row, row * p.rows_dim, 0}, {32, 32, 1, 1}});
        else
            st = encode(&m.out, {p.out, Element::kBf16, 2, {cols, static_cast<uint64_t>(p.groups.num_rows), 1, 1},
                                 {row, 0, 0}, {64, 32, 1, 1}});
    }
    m.residual = m.b;  // not used
    if (st == EP_OK && p.residual)
        st = encode(&m.residual, {p.residual, Element::kBf16, 2, {static_cast<uint64_t>(p.cols_dim), static_cast<uint64_t>(p.groups.num_rows), 1, 1},
                                  {static_cast<uint64_t>(p.residual_row_bytes), 0, 0}, {64, 32, 1, 1}});
    if (p.a_words) {
        m.a = m.a_small = m.b;  // not used
    } else {
        if (st == EP_OK) st = encode(&m.a, a);
        if (st == EP_OK) st = encode(&m.a_small, a_small);
    }
    if (st != EP_OK) return st;
    // A pair of CTAs computes 256 rows: each loads half of the weight tile, so that a row of products takes a
    // third less shared-memory fill.  Where the rows of a group would leave one of the two idle, single CTAs; in
    // FP8, where a block's sums wait for both CTAs of a pair, single CTAs up to 1024 rows.  Measured at 32 experts,
    // 4096 x 4096, single against pair: bf16 185 and 185 us at 128 rows an expert, 222 and 203 at 200, 1361 and
    // 1241 at 2048; FP8 106 and 125 at 128, 363 and 388 at 700, 567 and 557 at 1024, 1105 and 1034 at 2048.
    cudaError_t err;
    if (has_words(FORM) && p.a_words)
        err = launch_kernel(grouped_gemm_kernel<FORM, 1, has_words(FORM)>, dim3(h->plan.num_sms), dim3(kGemmThreads),
                            kMaxSmem, stream, 1, m, p);
    else if (pairs)
        err = launch_kernel(grouped_gemm_kernel<FORM, 2>, dim3(2 * most_pairs), dim3(kGemmThreads), kMaxSmem, stream,
                            2, m, p);
    else
        err = launch_kernel(grouped_gemm_kernel<FORM, 1>, dim3(h->plan.num_sms), dim3(kGemmThreads), kMaxSmem, stream, 1, m, p);
    if (err != cudaSuccess) return cuda_fail(err, "grouped product launch");
    return EP_OK;
}

// Checks that every form shares; fills the groups' part of the parameters.
ep_status check_groups(const ep_handle* h, int64_t num_rows, int32_t n, int32_t k, const int32_t* group_count,
                       const int32_t* group_begin, GemmParams* p) {
    if (h == nullptr) return fail(EP_ERR_INVALID_ARG, "handle is NULL");
    const ep_status st = check_group_args(h, num_rows, group_count, group_begin);
    if (st != EP_OK) return st;
    const int32_t groups = h->cfg.num_experts;
    EP_CHECK_ARG(n >= 8 && n % 8 == 0 && k >= 8 && k % 8 == 0, "n %d and k %d must be positive multiples of 8", n, k);
    // tiles are numbered in 32 bits
    const int64_t wide = n > k ? n : k;
    const int64_t row_tiles = (num_rows > wide * groups ? num_rows : wide * groups) / kTileRows + groups;
    if (row_tiles * (wide / kColBox + 1) >= (INT64_C(1) << 30))
        return fail(EP_ERR_UNSUPPORTED, "%lld rows by %lld columns need too many tiles", static_cast<long long>(num_rows),
                    static_cast<long long>(wide));
    p->groups = {group_count, group_begin, num_rows, static_cast<int32_t>(num_rows / groups), groups};
    p->status = h->status;
    p->wait_limit_ns = h->wait_limit_ns;
    return EP_OK;
}

// Of the parts of one wave of tiles.
int64_t parts_bytes(const ep_handle* h) { return static_cast<int64_t>(h->plan.num_sms) * kEpilogueWarps * kPartFloats * sizeof(float); }

bool row_stride_ok(int64_t bytes, int64_t least) { return bytes >= least && bytes % 16 == 0 && bytes < (INT64_C(1) << 40); }

bool rows_aligned32(const void* p, int64_t row_bytes) {
    return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && row_bytes % 32 == 0;
}

// The operands of a product of rows; fills the rows' and the output's part of the parameters.
ep_status check_rows(const void* x, int64_t x_row_bytes, int64_t x_least, const void* w, void* out, int64_t out_row_bytes,
                     int32_t n, GemmParams* p) {
    EP_CHECK_ARG(x && w && out && aligned4(x) && aligned16(w) && aligned16(out),
                 "x must be a 4-byte, w and out 16-byte aligned device pointers");
    EP_CHECK_ARG(x_row_bytes >= x_least && x_row_bytes % 4 == 0 && x_row_bytes < (INT64_C(1) << 40) &&
                     row_stride_ok(out_row_bytes, 2 * static_cast<int64_t>(n)),
                 "row strides must hold a row, in multiples of 4 (x %lld bytes) and 16 (out %lld)",
                 static_cast<long long>(x_row_bytes), static_cast<long long>(out_row_bytes));
    if (!aligned16(x) || x_row_bytes % 16 != 0) p->a_words = static_cast<const uint8_t*>(x);
    p->a_row_bytes = x_row_bytes;
    p->out = out;
    p->out_row_bytes = out_row_bytes;
    p->wide_stores = rows_aligned32(out, out_row_bytes);
    return EP_OK;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" {

ep_status ep_grouped_gemm(ep_handle* h, int64_t num_rows, int32_t n, int32_t k, const int32_t* group_count,
                          const int32_t* group_begin, const void* x, int64_t x_row_bytes, const void* w,
                          int32_t w_transposed, void* out, int64_t out_row_bytes, int64_t expected_rows,
                          ep_stream_t stream) {
    EP_TRACE();
    GemmParams p = {};
    const ep_status st = check_groups(h, num_rows, n, k, group_count, group_begin, &p);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(expected_rows >= 0, "expected_rows %lld < 0", static_cast<long long>(expected_rows));
    if (num_rows == 0) return EP_OK;
    const ep_status rows = check_rows(x, x_row_bytes, 2 * static_cast<int64_t>(k), w, out, out_row_bytes, n, &p);
    if (rows != EP_OK) return rows;
    p.cols_dim = n;
    p.contraction = k;
    const int64_t rows_each = expected_rows ? expected_rows : num_rows / p.groups.groups;
    const int groups = p.groups.groups;
    const Operand a = row_operand(x, false, k, num_rows, x_row_bytes, kBox);
    const Operand a_small = row_operand(x, false, k, num_rows, x_row_bytes, kRowBox);
    if (!w_transposed)
        return launch<kForward>(h, a, a_small, weight_operand(w, false, k, n, groups, kBox),
                                weight_operand(w, false, k, n, groups, kColBox), p, rows_each, stream);
    p.b_chunked = chunked_columns(n);
    return launch<kTransposed>(h, a, a_small, weight_across_operand(w, n, k, groups, p.b_chunked ? kBox / 64 : 1),
                               weight_across_operand(w, n, k, groups, 1), p, rows_each, stream);
}

int64_t ep_grouped_gemm_act_workspace(const ep_handle* h, int64_t num_rows, int32_t n, int32_t k, int32_t gated, int64_t expected_rows) {
    if (h == nullptr || num_rows <= 0 || n <= 0 || k < 2 * kLeastPartSteps * 64) return 0;
    // wide tiles leave half of the CTAs without one, or more
    const int64_t rows_each = expected_rows > 0 ? expected_rows : num_rows / h->cfg.num_experts;
    const int32_t width = gated ? n / 2 : n, cols = gated ? kMaxTileCols / 2 : kMaxTileCols;
    const int64_t tiles = h->cfg.num_experts * ((rows_each + kTileRows - 1) / kTileRows) * ((width + cols - 1) / cols);
    return 2 * tiles <= h->plan.num_sms ? parts_bytes(h) : 0;
}

ep_status ep_grouped_gemm_act(ep_handle* h, int64_t num_rows, int32_t n, int32_t k, const int32_t* group_count,
                              const int32_t* group_begin, const void* x, int64_t x_row_bytes, const void* w,
                              const float* bias, int32_t act, int32_t gated, const float* row_weights, const void* residual,
                              int64_t residual_row_bytes, void* pre, int64_t pre_row_bytes, void* out, ep_dtype out_dtype,
                              int64_t out_row_bytes, int64_t expected_rows, void* workspace, int64_t workspace_bytes,
                              ep_stream_t stream) {
    EP_TRACE();
    GemmParams p = {};
    const ep_status st = check_groups(h, num_rows, n, k, group_count, group_begin, &p);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(!gated || n % 16 == 0, "gated: n %d must be two widths of a multiple of 8", n);
    EP_CHECK_ARG(act >= EP_ACT_NONE && act <= EP_ACT_GELU, "act %d is no activation", act);
    EP_CHECK_ARG(out_dtype == EP_BF16 || (out_dtype == EP_FP32 && !gated), "out_dtype must be EP_BF16, or EP_FP32 where it is not gated");
    EP_CHECK_ARG(expected_rows >= 0, "expected_rows %lld < 0", static_cast<long long>(expected_rows));
    if (num_rows == 0) return EP_OK;
    const int32_t width = gated ? n / 2 : n;
    p.out_fp32 = out_dtype == EP_FP32;
    const ep_status rows = check_rows(x, x_row_bytes, 2 * static_cast<int64_t>(k), w, out, out_row_bytes, p.out_fp32 ? 2 * width : width, &p);
    if (rows != EP_OK) return rows;
    EP_CHECK_ARG(p.a_words == nullptr, "x must be 16-byte aligned, its rows multiples of 16 bytes apart (%lld)", static_cast<long long>(x_row_bytes));
    EP_CHECK_ARG(aligned16(bias) && aligned4(row_weights), "bias must be 16-byte aligned, row_weights 4-byte aligned");
    EP_CHECK_ARG(!residual || (aligned16(residual) && row_stride_ok(residual_row_bytes, 2 * static_cast<int64_t>(width))),
                 "residual must be 16-byte aligned with a row stride in multiples of 16 that holds a row (%lld bytes)",
                 static_cast<long long>(residual_row_bytes));
    EP_CHECK_ARG(!pre || (aligned16(pre) && row_stride_ok(pre_row_bytes, 2 * static_cast<int64_t>(n))),
                 "pre must be 16-byte aligned with a row stride in multiples of 16 that holds a row (%lld bytes)",
                 static_cast<long long>(pre_row_bytes));
    p.cols_dim = width;
    p.contraction = k;
    p.bias = bias;
    p.act = act;
    p.row_weights = row_weights;
    p.residual = static_cast<const uint8_t*>(residual);
    p.residual_row_bytes = residual_row_bytes;
    p.pre = static_cast<uint8_t*>(pre);
    p.pre_row_bytes = pre_row_bytes;
    const int64_t need = ep_grouped_gemm_act_workspace(h, num_rows, n, k, gated, expected_rows);
    EP_CHECK_ARG(!workspace || need == 0 || (aligned16(workspace) && workspace_bytes >= need),
                 "workspace must be 16-byte aligned and hold %lld bytes, got %lld", static_cast<long long>(need), static_cast<long long>(workspace_bytes));
    if (need > 0) p.parts = static_cast<float*>(workspace);
    p.tickets = h->part_tickets;
    p.pre_wide = pre && rows_aligned32(pre, pre_row_bytes) && (!gated || width % 16 == 0);
    const int64_t rows_each = expected_rows ? expected_rows : num_rows / p.groups.groups;
    const int groups = p.groups.groups;
    const Operand a = row_operand(x, false, k, num_rows, x_row_bytes, kBox);
    const Operand a_small = row_operand(x, false, k, num_rows, x_row_bytes, kRowBox);
    const Operand b = weight_operand(w, false, k, n, groups, kBox), b_small = weight_operand(w, false, k, n, groups, kColBox);
    if (p.out_fp32) return launch<kActivatedFp32>(h, a, a_small, b, b_small, p, rows_each, stream);
    return gated ? launch<kGated>(h, a, a_small, b, b_small, p, rows_each, stream)
                 : launch<kActivated>(h, a, a_small, b, b_small, p, rows_each, stream);
}

ep_status ep_grouped_gemm_wgrad(ep_handle* h, int64_t num_rows, int32_t n, int32_t k, const int32_t* group_count,
                                const int32_t* group_begin, const void* dy, int64_t dy_row_bytes, const void* x,
                                int64_t x_row_bytes, void* dw, ep_dtype dw_dtype, int32_t accumulate,
                                ep_stream_t stream) {
    EP_TRACE();
    GemmParams p = {};
    const ep_status st = check_groups(h, num_rows, n, k, group_count, group_begin, &p);
    if (st != EP_OK) return st;
    EP_CHECK_ARG(dw_dtype == EP_FP32 || dw_dtype == EP_BF16, "dw_dtype must be EP_FP32 or EP_BF16");
    EP_CHECK_ARG(!accumulate || dw_dtype == EP_FP32, "accumulate needs an fp32 dw");
    EP_CHECK_ARG(dw && aligned16(dw), "dw must be a 16-byte aligned device pointer");
    if (num_rows == 0) {
        if (accumulate) return EP_OK;
        DeviceGuard guard(h->device);
        const size_t bytes = static_cast<size_t>(p.groups.groups) * n * k * (dw_dtype == EP_FP32 ? 4 : 2);
        const cudaError_t err = cudaMemsetAsync(dw, 0, bytes, stream);
        return err == cudaSuccess ? EP_OK : cuda_fail(err, "clearing dw");
    }
    EP_CHECK_ARG(dy && x && aligned16(dy) && aligned16(x), "dy and x must be 16-byte aligned device pointers");
    EP_CHECK_ARG(row_stride_ok(x_row_bytes, 2 * static_cast<int64_t>(k)) &&
                     row_stride_ok(dy_row_bytes, 2 * static_cast<int64_t>(n)),
                 "row strides must be multiples of 16 that hold a row (x %lld, dy %lld bytes)",
                 static_cast<long long>(x_row_bytes), static_cast<long long>(dy_row_bytes));
    p.rows_dim = n;
    p.cols_dim = k;
    p.out = dw;
    p.out_fp32 = dw_dtype == EP_FP32;
    p.accumulate = accumulate != 0;
    p.out_row_bytes = static_cast<int64_t>(k) * (p.out_fp32 ? 4 : 2);
    p.wide_stores = rows_aligned32(dw, p.out_row_bytes);
    p.a_chunked = chunked_columns(n);
    p.b_chunked = chunked_columns(k);
    return launch<kWeightGrad>(h, across_operand(dy, n, num_rows, dy_row_bytes, p.a_chunked ? kBox / 64 : 1),
                               across_operand(dy, n, num_rows, dy_row_bytes, 1),
                               across_operand(x, k, num_rows, x_row_bytes, p.b_chunked ? kBox / 64 : 1),
                               across_operand(x, k, num_rows, x_row_bytes, 1), p, n, stream);
}

ep_status ep_grouped_gemm_fp8(ep_handle* h, int64_t num_rows, int32_t n, int32_t k, const int32_t* group_count,
                              const int32_t* group_begin, const void* x, int64_t x_row_bytes, const void* x_scales,
                              int64_t x_scale_row_bytes, int32_t scales_ue8m0, const void* w, const float* w_scales,
                              void* out, int64_t out_row_bytes, int64_t expected_rows, ep_stream_t stream) {
    EP_TRACE();
    GemmParams p = {};
    const ep_status st = check_groups(h, num_rows, n, k, group_count, group_begin, &p);
    if (st != EP_OK) return st;
    if (k % kFp8Group != 0) return fail(EP_ERR_UNSUPPORTED, "FP8 products need k %% 128 == 0 (k %d)", k);
    EP_CHECK_ARG(expected_rows >= 0, "expected_rows %lld < 0", static_cast<long long>(expected_rows));
    if (num_rows == 0) return EP_OK;
    const ep_status rows = check_rows(x, x_row_bytes, k, w, out, out_row_bytes, n, &p);
    if (rows != EP_OK) return rows;
    const int64_t scale_row = static_cast<int64_t>(k / kFp8Group) * (scales_ue8m0 ? 1 : 4);
    EP_CHECK_ARG(x_scales && w_scales && aligned4(w_scales) && x_scale_row_bytes >= scale_row &&
                     (scales_ue8m0 || (aligned4(x_scales) && x_scale_row_bytes % 4 == 0)),
                 "x_scales or w_scales missing or misaligned, or x_scale_row_bytes %lld too small",
                 static_cast<long long>(x_scale_row_bytes));
    p.cols_dim = n;
    p.contraction = k;
    p.x_scales = static_cast<const uint8_t*>(x_scales);
    p.x_scale_row_bytes = x_scale_row_bytes;
    p.scales_ue8m0 = scales_ue8m0 != 0;
    p.w_scales = w_scales;
    const int64_t rows_each = expected_rows ? expected_rows : num_rows / p.groups.groups;
    return launch<kFp8>(h, row_operand(x, true, k, num_rows, x_row_bytes, kBox),
                        row_operand(x, true, k, num_rows, x_row_bytes, kRowBox),
                        weight_operand(w, true, k, n, p.groups.groups, kBox),
                        weight_operand(w, true, k, n, p.groups.groups, kColBox), p, rows_each, stream);
}

}  // extern "C"
