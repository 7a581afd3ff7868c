// Block-scaled FP8 matrix product, dense and per expert on ragged row groups.
//
// Source: "Practical FP4 Training for Large-Scale MoE Models on Hopper GPUs",
// technical overview section 2 (items 1-3): E4M3 operands with 128-element
// blocks and FP32 block scales feed the expert products, whose token groups
// are ragged and unpadded.
//
//   C[m, n] = sum_b sa[m, b] * sb[n, b] * ( sum_{k in block b} A[m, k] B[n, k] )
//
// b runs over the 128-element blocks of K.  The inner sums are tensor-core
// products (kind::f8f6f4, FP32 accumulation); the outer sum is kept in FP32
// registers: one multiply sa * sb per row and block and one FMA per element.
//
// The kernels are templates over what becomes of a finished sum (Epi): written
// as it is, with a bias, an activation and a residual, as the product of an
// activated and a plain projection, or as the gradient of an activation.
#pragma once

#include <type_traits>

#include "fq_epilogue.cuh"
#include "fq_tc.cuh"

namespace fq {

namespace {

constexpr int kRowsM = 128;       // rows of c of a CTA (its TMEM lanes)
constexpr int kBlockK = 128;      // one scale block, one pipeline stage
constexpr int kPromoteWarps = 8;  // two warpgroups
constexpr int kMmThreads = (kPromoteWarps + 4) * 32;
// Registers of a promoting and of another thread: 384 threads x 168 at launch =
// 64512 = 256 x 200 + 128 x 104 = 256 x 208 + 128 x 88.  The other roles' spills
// cost 10 to 20 % (at 56); with a scale per column the promoting warps need more
// (with an epilogue they do not: act without options, 65536 x 2048 x 7168, 748 us at 200,
// 779 at 208).  What is spilled all the same, bytes stored by -Xptxas -v, in tiles of pairs:
// act up to 4, gated products 4 to 12 (up to 76 loaded, in the loop's scales), gradients 28 to
// 60, gated gradients 28 to 32, and 144 to 148 with a scale per column (65536 x 2048 x 7168 with
// h 2154 us, the plain activation's gradient 1379).
constexpr int promote_regs(bool col_scale) { return col_scale ? 208 : 200; }
constexpr int other_regs(bool col_scale) { return col_scale ? 88 : 104; }
constexpr int kRaster = 8;        // row tiles walked together over the columns
constexpr int kScaleBlocks = 4;   // blocks whose scales are fetched together
constexpr int kBoxCols = 32;      // columns of c that a warp writes at once
constexpr int kNotes = 8;         // tiles worked out together (NoteWalk)

// What the second operand's scales and the tiles are:
//   kTileScale  forward, one scale per 128x128 weight tile
//   kRowScale   forward, one scale per weight row and block
//   kWgrad      weight gradient: per group, sum over its 128-token blocks of
//               products of transposed operands, both with a scale per row
//               and block
enum Mode { kTileScale, kRowScale, kWgrad };

// What c is.
enum Out { kBf16, kF32, kE4m3 };

// What becomes of a finished sum v (of the two of an output, for kGated):
//   kPlain      c = v
//   kAct        c = residual + act(v + bias)
//   kGated      c = act(gate) * up
//   kActGrad    c = v * act'(z)
//   kGatedGrad  c = (v * up * act'(gate), v * act(gate)) of z = (gate, up)
enum Epi { kPlain, kAct, kGated, kActGrad, kGatedGrad };

// Boxes of 32 rows x kBoxCols columns of c, staged by a warp.
template <bool kWide>
struct Box {
    static constexpr int row = kBoxCols * (kWide ? 4 : 2);
    static constexpr int bytes = 32 * row;
};

// kCtas CTAs work on a tile of 128 kCtas rows.  Columns of the tile: 256 for a
// pair, 128 for one CTA.  Gated: 256 columns are 128 of c, each half of the
// accumulator 64 gate columns and the up columns beside them, so that a thread
// holds both sums of an output; 128 columns of c for one CTA too, so that a tile
// holds whole 128-element blocks of a quantized output.
template <int kCtas, Out kOut, Epi kEpi>
struct Shape {
    static constexpr bool gated = kEpi == kGated;
    static constexpr int bn = gated ? 256 : 128 * kCtas;
    static constexpr int step = gated ? 128 : bn;     // columns of c
    static constexpr int cols = bn / 2;               // of a promoting thread
    static constexpr int a_bytes = kRowsM * kBlockK;  // of a stage of a CTA
    static constexpr int b_rows = bn / kCtas;
    static constexpr int b_bytes = b_rows * kBlockK;
    static constexpr int box_rows = gated ? 64 : b_rows;  // of a tensor copy of b
    // Boxes that a promoting warp uses in turn; an input of c's type is fetched into
    // them ahead of its use.  Behind them, where the epilogue has an input, a BF16 box
    // for what goes out beside c, and for gradients in FP32 two for z.
    static constexpr bool inputs = kEpi == kAct || kEpi == kActGrad || kEpi == kGatedGrad;
    static constexpr bool fetches = inputs && (kEpi == kAct || kOut == kBf16);
    static constexpr int box_bytes = Box<kOut == kF32>::bytes;
    static constexpr int boxes = kEpi == kPlain   ? (kOut == kF32 ? 1 : 2)
                                 : kEpi == kAct   ? (kOut == kF32 ? 2 : 3)
                                 : kEpi != kGated ? (kOut == kF32 ? 2 : 4)
                                 : kOut == kF32   ? 3
                                                  : (kCtas == 1 ? 4 : 5) - (kOut == kE4m3 ? 1 : 0);
    static constexpr int parts = kEpi == kGatedGrad ? 2 : 1;  // matrices of the input and c
    static constexpr int slots = boxes / parts;               // steps whose boxes they are
    static constexpr int extra = !inputs ? 0 : (fetches ? 1 : 3);  // BF16 boxes
    static constexpr int warp_bytes = boxes * box_bytes + extra * Box<false>::bytes;
    static constexpr int stages =
        kEpi == kPlain ? 5
                       : (b_rows > 128 ? 3 : 4) - (kOut == kF32 ? 1 : 0);
};

// Shared memory behind the operand stages and the staged output.
template <int kCtas, Out kOut, Epi kEpi>
struct MmTail {
    using S = Shape<kCtas, kOut, kEpi>;
    uint64_t full[S::stages], empty[S::stages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t scale_full[2], scale_empty[2];
    uint32_t tmem;
    int32_t abort;
    // column scales of two groups of kScaleBlocks blocks
    alignas(16) float col_scale[2][kScaleBlocks][S::bn];
    // largest magnitude of a row in each half of a 128-column block
    uint32_t row_max[kOut == kE4m3 ? 2 : 1][2][kOut == kE4m3 ? kRowsM : 1];
    uint64_t in_full[kPromoteWarps][S::slots];
    // the bias of a promoting warp's columns
    alignas(16) float bias[kEpi == kAct ? kPromoteWarps : 1][kEpi == kAct ? S::cols : 4];
    // its next tiles
    int4 notes[kEpi == kPlain ? 1 : kPromoteWarps][kNotes];
    // int32 off[G + 2], first[G + 2] follow
};

struct MmArgs {
    const float *sa, *sb;
    const int64_t *offs;
    void *c;
    int32_t *dev_status;
    int32_t G;
    int32_t M;        // tokens
    int32_t R, N;     // rows (weight gradient only) and columns of c
    int32_t KB;       // 128-element blocks of K (forward only)
    int32_t sb_rows;  // rows of sb per group (forward only)
    int32_t add;      // weight gradient: c += instead of c =
    EpiArgs e;
};

// Tensor maps: operands, c, z (or h) beside it, the epilogue's input.
struct MmMaps {
    CUtensorMap a, b, c, d, in;
};

// One output tile.
struct Tile {
    int32_t g;          // group
    int32_t row, n0;    // first row and column in c (row: in the group's matrix for kWgrad)
    int32_t end;        // rows of c end here
    int32_t blocks;     // blocks to add up
    int32_t xblk;       // first block's index along K
    int32_t arow, brow; // operand rows
};

// Row tile, column tile of the tile index: kRaster row tiles share a walk over
// the columns, so that the operands of the tiles in flight stay in L2.
__device__ __forceinline__ void tile_coords(int32_t idx, int32_t mt, int32_t nt, int32_t &i,
                                            int32_t &j)
{
    const int32_t band = idx / (kRaster * nt);
    const int32_t rows = min(kRaster, mt - band * kRaster);
    const int32_t r = idx - band * kRaster * nt;
    j = r / rows;
    i = band * kRaster + r - j * rows;
}

template <Mode kMode, int kRows, int kStep, int kParts>
__device__ __forceinline__ Tile tile_at(int32_t idx, const MmArgs &p, const int32_t *off,
                                        const int32_t *first, int32_t mt, int32_t nt)
{
    Tile t;
    int32_t i, j;
    if (kMode == kWgrad) {
        t.g = idx / (mt * nt);
        tile_coords(idx - t.g * mt * nt, mt, nt, i, j);
        t.row = t.arow = i * kRows;
        t.n0 = t.brow = j * kStep;
        t.end = p.R;
        t.blocks = first[t.g + 1] - first[t.g];
        t.xblk = first[t.g];
    } else {
        tile_coords(idx, mt, nt, i, j);
        t.g = group_of_tile(first, p.G + 1, i);
        t.row = t.arow = off[t.g] + (i - first[t.g]) * kRows;
        t.n0 = j * kStep;
        t.brow = t.g * kParts * p.N + t.n0;
        t.end = off[t.g + 1];
        t.blocks = t.g < p.G ? p.KB : 0;  // rows of no group are 0
        t.xblk = 0;
    }
    return t;
}

// Byte of 16-byte piece i of row r in a box: the swizzle of a tensor copy of
// rows of 64 (BF16) or 128 (FP32) bytes.
template <bool kWide>
__device__ __forceinline__ int box_at(int r, int i)
{
    return Box<kWide>::row * r + 16 * (kWide ? i ^ (r & 7) : i ^ ((r >> 1) & 3));
}

// A warp's box, from registers (lane l holds row l, packed pairs of columns).
template <bool kWide>
__device__ __forceinline__ void stage_box(uint8_t *box, const uint64_t *acc)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < Box<kWide>::row / 16; i++) {
        uint4 *to = reinterpret_cast<uint4 *>(box + box_at<kWide>(lane, i));
        float v[8];
        if (kWide) {
            unpack2(acc[2 * i], v[0], v[1]);
            unpack2(acc[2 * i + 1], v[2], v[3]);
            *to = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                             __float_as_uint(v[3]));
        } else {
#pragma unroll
            for (int h = 0; h < 4; h++)
                unpack2(acc[4 * i + h], v[2 * h], v[2 * h + 1]);
            *to = make_uint4(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]),
                             cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
        }
    }
}

// The staged box by ordinary stores, a row at a time: where the group's rows end
// inside the box, where rows of c (of `pitch` elements, columns from `limit` on are
// not written) are not 16-byte aligned, and for c += box, whose
// loads are waited for one by one (65536 tokens, 32 x 2048 x 7168: 1511 -> 7075 us).
template <bool kWide, bool kAdd>
__device__ __forceinline__ void store_box(void *c, const uint8_t *box, int64_t row0, int32_t rows,
                                          int32_t col, int32_t limit, int64_t pitch)
{
    const int e = threadIdx.x & 31, b = e * (kWide ? 4 : 2);
    if (col + e >= limit)
        return;
    for (int r = 0; r < rows; r++) {
        const uint8_t *from = box + box_at<kWide>(r, b >> 4) + (b & 15);
        const int64_t at = (row0 + r) * pitch + col + e;
        if (kWide) {
            float v = *reinterpret_cast<const float *>(from);
            if (kAdd)
                v += static_cast<float *>(c)[at];
            static_cast<float *>(c)[at] = v;
        } else {
            static_cast<uint16_t *>(c)[at] = *reinterpret_cast<const uint16_t *>(from);
        }
    }
}

// acc += the BF16 values c holds (before the one rounding).  Two bytes a lane from
// as many rows (the case above: 1460 -> 3431 us).
template <int kCols>
__device__ __forceinline__ void add_bf16(const void *c, int64_t row_off, int32_t col, int32_t N,
                                         uint64_t *acc)
{
#pragma unroll
    for (int i = 0; i < kCols / 2; i++) {
        float v[2];
        unpack2(acc[i], v[0], v[1]);
#pragma unroll
        for (int h = 0; h < 2; h++)
            if (col + 2 * i + h < N)
                v[h] += bf16_lo(static_cast<const uint16_t *>(c)[row_off + col + 2 * i + h]);
        acc[i] = pack2(__float_as_uint(v[0]), __float_as_uint(v[1]));
    }
}

// The end of a tile: what a warp makes of its 32 rows and S::cols columns of sums
// (lane l holds row l, packed pairs of columns) and writes, a step of 32 columns at
// a time, by way of its boxes in shared memory.  They are used in turn: the n-th
// output of the warp, over all tiles, goes through box n mod S::boxes.  An input
// (residual or z) is fetched into the box that the output of its place goes out
// from: in the middle of a step, when the boxes of the step before have been read,
// they take the next inputs, those of the next tile at the end of this.  Between
// tiles nothing is kept but two counts: the sums need the registers.
//
// This is run once a tile by two warps a scheduler, so that latency is what it
// costs, that of fetching instructions above all: a taken branch costs some 100
// cycles, also one over code that is not wanted or back to a loop's start.  So the
// code is straight, once for each form of the activation (Form), and options are
// predicates in it; what a tile at the end of a group or of the columns needs, or
// rows that are not 16-byte aligned, is done at a step's begin and end, behind one
// vote each; and all single-thread work is in elected blocks.  16384 x 7168 x 2048
// with bias, silu, residual and z: 335 us, with silu alone 281; without any option
// 216 (the plain product 206 to 223).
template <int kCtas, Mode kMode, Out kOut, Epi kEpi>
struct Finish {
    using S = Shape<kCtas, kOut, kEpi>;
    static constexpr int kCols = S::cols;
    static constexpr bool kWideOut = kOut == kF32;
    static constexpr uint32_t kParts = S::parts;
    static constexpr uint32_t kBoxes = S::boxes;
    static constexpr unsigned kAll = 0xffffffffu;

    const MmArgs &p;
    const MmMaps &maps;
    uint8_t *stage;
    uint64_t *in_full;  // a barrier for a step's boxes: a phase for each of their uses
    uint32_t n, asked;  // boxes used, and taken for inputs
    const float *bias;  // in shared memory
    int lane;
    bool fetch;            // whether inputs come by tensor copies
    bool odd;              // whether the tile is not 32 whole rows and S::cols whole columns
    int32_t row0, end, g;  // of the tile

    __device__ __forceinline__ Finish(const MmArgs &args, const MmMaps &m, uint8_t *boxes,
                                      uint64_t *full, const float *b, uint32_t used,
                                      uint32_t taken)
        : p(args), maps(m), stage(boxes), in_full(full), n(used), asked(taken), bias(b),
          lane(fresh_tid() & 31)
    {
        fetch = S::fetches && p.e.in &&
                vector(kWideOut ? 4 : 2, static_cast<int64_t>(kParts) * p.N, p.N);
    }

    __device__ __forceinline__ int32_t rows() const { return min(32, end - row0); }
    __device__ __forceinline__ uint8_t *box_of(uint32_t i) const
    {
        return stage + i % kBoxes * S::box_bytes;
    }
    // Whether columns [first, first + limit) of a matrix of `pitch` elements can be
    // copied in 16-byte pieces.
    static __device__ __forceinline__ bool vector(int32_t size, int64_t pitch, int32_t first)
    {
        return pitch * size % 16 == 0 && static_cast<int64_t>(first) * size % 16 == 0;
    }
    // Boxes of the tile at these rows and columns (not for gated results).
    __device__ __forceinline__ uint32_t boxes_of(int32_t row, int32_t last, int32_t col) const
    {
        return row < last && col < p.N ? (min(p.N - col, kCols) + 31) / 32 * kParts : 0;
    }

    // ---- inputs

    // Boxes up to n have been read: they take the inputs of this tile (`all` boxes from
    // box n0 on, columns from col0) and of the next (next_all boxes).
    __device__ __forceinline__ void ask(uint32_t n0, uint32_t all, int32_t col0, uint32_t next_all,
                                        int32_t next_row, int32_t next_col)
    {
        if (!S::fetches || !fetch)
            return;
        const uint32_t to = min(n + kBoxes, n0 + all + next_all);
        if (elect_one()) {
            tma_store_wait_read<0>();
            for (uint32_t i = asked; i < to; i += kParts) {
                const bool next = i - n0 >= all;
                const int32_t step = (next ? i - n0 - all : i - n0) / kParts;
                uint64_t *bar = in_full + i / kParts % S::slots;
                mbar_arrive_expect_tx(bar, kParts * S::box_bytes);
#pragma unroll
                for (uint32_t q = 0; q < kParts; q++)
                    tma_load_2d(box_of(i + q), &maps.in,
                                q * p.N + (next ? next_col : col0) + 32 * step,
                                next ? next_row : row0, bar);
            }
        }
        __syncwarp();
        asked = to;
    }

    // ---- columns

    // Eight columns of the lane's row, in pairs: the h-th eight of a box.
    template <bool kWide>
    static __device__ __forceinline__ void put8(uint8_t *box, int h, int lane, const uint64_t *v)
    {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; i++)
            unpack2(v[i], f[2 * i], f[2 * i + 1]);
        if (kWide) {
#pragma unroll
            for (int i = 0; i < 2; i++)
                *reinterpret_cast<uint4 *>(box + box_at<true>(lane, 2 * h + i)) =
                    make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                               __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
        } else {
            *reinterpret_cast<uint4 *>(box + box_at<false>(lane, h)) =
                make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                           cvt_bf16x2(f[6], f[7]));
        }
    }
    // The pairs in 16 bytes.
    template <bool kWide>
    static __device__ __forceinline__ void spread(const uint4 &w, uint64_t *v)
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        if (kWide) {
            v[0] = pack2(u[0], u[1]);
            v[1] = pack2(u[2], u[3]);
        } else {
#pragma unroll
            for (int h = 0; h < 4; h++)
                v[h] = pack2f(bf16_lo(u[h]), bf16_hi(u[h]));
        }
    }
    // ---- what is behind the boxes

    __device__ __forceinline__ uint8_t *side_box() const { return stage + kBoxes * S::box_bytes; }
    // The box that the part's input is read from in this step.
    __device__ __forceinline__ uint8_t *in_box(uint32_t part) const
    {
        return S::fetches ? box_of(n + part)
                          : side_box() + (1 + part) * static_cast<uint32_t>(Box<false>::bytes);
    }
    // A step's input where it does not come by a tensor copy, or is not to be used (rows
    // of no group, whose gradients are 0 with z = 0): a row at a time.
    __device__ __forceinline__ void fill(int32_t col) const
    {
        constexpr bool kWide = kWideOut && S::fetches;
        constexpr int kSize = kWide ? 4 : 2;
        const int b = lane * kSize;
        const bool none = kEpi != kAct && g == p.G;
#pragma unroll 1
        for (uint32_t q = 0; q < kParts; q++) {
            uint8_t *box = in_box(q);
            const uint8_t *from = static_cast<const uint8_t *>(p.e.in) +
                                  ((static_cast<int64_t>(row0) * kParts + q) * p.N + col + lane) * kSize;
            // half of the rows are on their way at once
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 16) {
                uint32_t v[16];
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const bool there = !none && r0 + r < rows() && col + lane < p.N;
                    const uint8_t *at = from + static_cast<int64_t>(r0 + r) * kParts * p.N * kSize;
                    v[r] = !there  ? 0u
                           : kWide ? *reinterpret_cast<const uint32_t *>(at)
                                   : *reinterpret_cast<const uint16_t *>(at);
                }
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    uint8_t *to = box + box_at<kWide>(r0 + r, b >> 4) + (b & 15);
                    if (kWide)
                        *reinterpret_cast<uint32_t *>(to) = v[r];
                    else
                        *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(v[r]);
                }
            }
        }
        __syncwarp();
    }

    // ---- outputs

    __device__ __forceinline__ void begin(int32_t row, int32_t last, int32_t group, int32_t col0,
                                          int32_t cols)
    {
        row0 = row;
        end = last;
        g = group;
        constexpr int kSize = kOut == kE4m3 ? 1 : (kWideOut ? 4 : 2);
        odd = __any_sync(kAll, rows() != 32 || col0 + cols > p.N || g == p.G ||
                                   !vector(kSize, p.N, 0) || (p.e.side && !vector(2, p.N, 0)));
    }
    // A box by ordinary stores, where its rows or columns end or are not aligned.
    template <bool kWide>
    __device__ __forceinline__ void box_rows(const uint8_t *box, void *c, int32_t col,
                                             int32_t first, int64_t pitch) const
    {
        store_box<kWide, false>(static_cast<uint8_t *>(c) + static_cast<int64_t>(first) * (kWide ? 4 : 2),
                                box, row0, rows(), col, p.N, pitch);
    }
    // A step's boxes, from box n on, go out: the projections of a gated result and c's.
    // The boxes of the next step are free then, if they are not inputs.
    __device__ __forceinline__ void send(int32_t col)
    {
        constexpr bool kFront = kEpi == kGated;
        constexpr uint32_t kC = kOut == kE4m3 ? 0 : kParts;
        constexpr int kFree = kFront ? 3 : kParts;  // boxes of a step
        const bool side = kFront && p.e.side != nullptr;
        const uint32_t c0 = n + (side ? 2 : 0);
        fence_async_shared();
        __syncwarp();
        if (__any_sync(kAll, odd)) {
            if (side)
#pragma unroll 1
                for (uint32_t q = 0; q < 2; q++)
                    box_rows<false>(box_of(n + q), p.e.side, col, q * p.N, 2 * static_cast<int64_t>(p.N));
#pragma unroll 1
            for (uint32_t q = 0; q < kC; q++)
                box_rows<kWideOut>(box_of(c0 + q), p.c, col, q * p.N, static_cast<int64_t>(kParts) * p.N);
            if (!kFront && p.e.side)
                box_rows<false>(side_box(), p.e.side, col, 0, p.N);
            __syncwarp();
        }
        if (elect_one()) {
            // a group for every box
            if (side)
#pragma unroll
                for (uint32_t q = 0; q < 2; q++) {
                    if (!odd)
                        tma_store_2d(&maps.d, box_of(n + q), q * p.N + col, row0);
                    tma_store_commit();
                }
#pragma unroll
            for (uint32_t q = 0; q < kC; q++) {
                if (!odd)
                    tma_store_2d(&maps.c, box_of(c0 + q), q * p.N + col, row0);
                tma_store_commit();
            }
            if (!S::fetches || !fetch)
                tma_store_wait_read<(kBoxes > kFree ? kBoxes - kFree : 0)>();
        }
        __syncwarp();
        n += kC + (side ? 2 : 0);
    }
    // Eight BF16 columns of the lane's row beside c, the h-th of a step: straight from
    // registers (boxes for them would take the place of inputs), or by way of their box.
    __device__ __forceinline__ void put_side(int h, int32_t col, const uint64_t *v) const
    {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; i++)
            unpack2(v[i], f[2 * i], f[2 * i + 1]);
        const uint4 w = make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]),
                                   cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
        uint16_t *to = static_cast<uint16_t *>(p.e.side) + static_cast<int64_t>(row0 + lane) * p.N + col;
        if (p.e.side && !odd)
            *reinterpret_cast<uint4 *>(to) = w;
        if (p.e.side && odd)
            *reinterpret_cast<uint4 *>(side_box() + box_at<false>(lane, h)) = w;
    }

    // ---- act(gate) * up

    // The projections and, unless it is quantized, the result go out; a quantized
    // one's 64 columns are left in acc, and their largest magnitude's bits (a NaN's are
    // the largest) are returned.
    template <bool kSigmoid>
    __device__ __forceinline__ uint32_t gated(uint64_t *acc, int32_t col0)
    {
        constexpr int kHalf = kCols / 4;  // pairs of the gate
        const Act act(p.e.act);
        const bool side = p.e.side != nullptr;
        uint32_t most = 0;
#pragma unroll
        for (int x = 0; x < kCols / 64; x++) {
            uint64_t *a = acc + 16 * x, *u = a + kHalf;
            const int32_t col = col0 + 32 * x;
            if (__any_sync(kAll, col >= p.N || rows() <= 0))
                break;
            uint8_t *gate_box = box_of(n), *up_box = box_of(n + 1);
            uint8_t *box = box_of(n + (side ? 2 : 0));
#pragma unroll
            for (int h = 0; h < 4; h++) {
                uint64_t v[4];
                const uint64_t *w = u + 4 * h;
                if (side) {
                    put8<false>(gate_box, h, lane, a + 4 * h);
                    put8<false>(up_box, h, lane, w);
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
                    v[i] = mul_x2(act.template value<kSigmoid>(a[4 * h + i]), w[i]);
                if (kOut == kE4m3) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        float f[2];
                        unpack2(v[i], f[0], f[1]);
                        most = max(most, max(__float_as_uint(f[0]) & 0x7FFFFFFFu,
                                             __float_as_uint(f[1]) & 0x7FFFFFFFu));
                        a[4 * h + i] = v[i];
                    }
                } else {
                    put8<kWideOut>(box, h, lane, v);
                }
            }
            if (kOut != kE4m3 || side)
                send(col);
        }
        return most;
    }
    __device__ __forceinline__ uint32_t gated(uint64_t *acc, int32_t col0)
    {
        return Act::sigmoid(p.e.act) ? gated<true>(acc, col0) : gated<false>(acc, col0);
    }
    // The lane's half of a block whose largest magnitude is `most`, as E4M3.
    __device__ __forceinline__ void quantized(const uint64_t *acc, int32_t col0, uint32_t most)
    {
        if (__any_sync(kAll, rows() <= 0))
            return;
        float r, s;
        const bool special = e4m3_factors(most, r, s);
        uint8_t *box = box_of(n++);
#pragma unroll
        for (int i = 0; i < kCols / 32; i++) {  // 16 codes a piece
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float v[4];
                unpack2(acc[8 * i + 2 * k], v[0], v[1]);
                unpack2(acc[8 * i + 2 * k + 1], v[2], v[3]);
                w[k] = cvt_e4m3x2(v[0] * r, v[1] * r) | cvt_e4m3x2(v[2] * r, v[3] * r) << 16;
                w[k] = special ? 0x7F7F7F7Fu : w[k];
            }
            *reinterpret_cast<uint4 *>(box + box_at<false>(lane, i)) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_async_shared();
        __syncwarp();
        if (col0 % 128 == 0 && lane < rows())
            p.e.scales[static_cast<int64_t>(row0 + lane) * (p.N / 128) + col0 / 128] = s;
        const bool whole = __all_sync(kAll, rows() == 32);
        if (!whole) {
            for (int k = lane; k < 4 * rows(); k += 32)
                *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.c) +
                                           static_cast<int64_t>(row0 + (k >> 2)) * p.N + col0 +
                                           16 * (k & 3)) =
                    *reinterpret_cast<const uint4 *>(box + box_at<false>(k >> 2, k & 3));
            __syncwarp();
        }
        if (elect_one()) {
            if (whole)
                tma_store_2d(&maps.c, box, col0, row0);
            tma_store_commit();
            tma_store_wait_read<(kBoxes > 3 ? kBoxes - 3 : 0)>();
        }
        __syncwarp();
    }

    // ---- eight columns of the others, the h-th of a step

    // The forms that have code of their own: the sums alone or with a residual, and
    // whatever there is besides (bias, z or h, relu), with sigmoids or without.  kSum is
    // for weights with a scale a block: 16384 x 7168 x 2048, without options 240 -> 222
    // us, with the residual 264 -> 246 (and 1 or 2 % more time for the forms beside it,
    // the code being longer); with a scale a row the main loop takes longer than the
    // end of the tile before, and it gained nothing.
    enum Form { kSum, kAny, kAnySigmoid };

    // c = residual + act(v + bias), z beside it
    template <Form kForm>
    __device__ __forceinline__ void activated(const uint64_t *a, int h, int32_t col,
                                              const float *b, const Act &act) const
    {
        constexpr int kPieces = kWideOut ? 2 : 1;
        uint8_t *box = box_of(n);
        uint64_t v[4], w[4];
        if (kForm != kSum) {
            float4 lo = {}, hi = {};
            if (p.e.bias) {
                lo = *reinterpret_cast<const float4 *>(b);
                hi = *reinterpret_cast<const float4 *>(b + 4);
            }
            v[0] = add_x2(a[0], pack2f(lo.x, lo.y));
            v[1] = add_x2(a[1], pack2f(lo.z, lo.w));
            v[2] = add_x2(a[2], pack2f(hi.x, hi.y));
            v[3] = add_x2(a[3], pack2f(hi.z, hi.w));
            put_side(h, col, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
                v[i] = a[i];
        }
#pragma unroll
        for (int i = 0; i < kPieces; i++) {
            uint4 piece = make_uint4(0, 0, 0, 0);
            if (p.e.in)
                piece = *reinterpret_cast<const uint4 *>(box + box_at<kWideOut>(lane, kPieces * h + i));
            spread<kWideOut>(piece, w + 2 * i);
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = add_x2(kForm == kSum ? v[i] : act.template value<kForm == kAnySigmoid>(v[i]),
                          w[i]);
        put8<kWideOut>(box, h, lane, v);
    }
    // The gradients of z, the activated value beside them.
    template <Form kForm>
    __device__ __forceinline__ void gradient(const uint64_t *a, int q, int32_t col, const Act &act) const
    {
        // d: the gradient of z or gate; x: of up; h: the activated value
        uint64_t d[4], x[4], h[4];
        spread<false>(*reinterpret_cast<const uint4 *>(in_box(0) + box_at<false>(lane, q)), x);
        if (kParts == 2)
            spread<false>(*reinterpret_cast<const uint4 *>(in_box(1) + box_at<false>(lane, q)), h);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            uint64_t slope;
            const uint64_t value = act.template gradient<kForm == kAnySigmoid>(x[i], slope);
            if (kParts == 2) {
                x[i] = mul_x2(a[i], value);
                d[i] = mul_x2(a[i], mul_x2(h[i], slope));
                h[i] = mul_x2(value, h[i]);
            } else {
                d[i] = mul_x2(a[i], slope);
                h[i] = value;
            }
        }
        put8<kWideOut>(box_of(n), q, lane, d);
        if (kParts == 2)
            put8<kWideOut>(box_of(n + 1), q, lane, x);
        put_side(q, col, h);
    }

    // The tile's columns from col0 on, kBody of them in a loop's body; the sums of the
    // next body move to where the last's were.
    template <Form kForm, int kBody>
    __device__ __forceinline__ void columns(uint64_t *acc, int32_t col0, uint32_t next_all,
                                            int32_t next_row, int32_t next_col,
                                            volatile int32_t *abort)
    {
        const uint32_t n0 = n, all = boxes_of(row0, end, col0);
        const bool fills = p.e.in && (!fetch || (kEpi != kAct && g == p.G));
        const Act act(p.e.act);
#pragma unroll 1
        for (int32_t at = col0; at < col0 + kCols; at += kBody) {
#pragma unroll
            for (int x = 0; x < kBody / 32; x++) {
                if (__any_sync(kAll, n - n0 >= all))
                    return;
                if (S::fetches && fetch)
                    warp_wait(smem_u32(in_full + n / kParts % S::slots), n / kParts / S::slots & 1,
                              abort);
                if (__any_sync(kAll, fills))
                    fill(at + 32 * x);
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    const int32_t col = at + 32 * x + 8 * h;
                    if constexpr (kEpi == kAct)
                        activated<kForm>(acc + 16 * x + 4 * h, h, col, bias + (col - col0), act);
                    else
                        gradient<kForm>(acc + 16 * x + 4 * h, h, col, act);
                    if (h == 1)
                        ask(n0, all, col0, next_all, next_row, next_col);
                }
                send(at + 32 * x);
            }
            if (kBody < kCols)
#pragma unroll
                for (int i = 0; i + kBody / 2 < kCols / 2; i++)
                    acc[i] = acc[i + kBody / 2];
        }
    }
    // next_row, next_last, next_col: where the next tile is (no rows: there is none).
    __device__ __forceinline__ void store(uint64_t *acc, int32_t col0, int32_t next_row,
                                          int32_t next_last, int32_t next_col,
                                          volatile int32_t *abort)
    {
        if constexpr (kEpi == kGated) {
            gated(acc, col0);
        } else {
            constexpr int kBody = kEpi == kAct ? kCols : (kCols < 64 ? kCols : 64);
            const uint32_t next_all = boxes_of(next_row, next_last, next_col);
            const auto run = [&](auto form) {
                columns<decltype(form)::value, kBody>(acc, col0, next_all, next_row, next_col, abort);
            };
            const bool sum = kEpi == kAct && kMode == kTileScale && !p.e.bias && !p.e.side &&
                             p.e.act == FQ_ACT_NONE;
            if (sum) {
                if constexpr (kEpi == kAct && kMode == kTileScale)
                    run(std::integral_constant<Form, kSum>{});
            } else if (Act::sigmoid(p.e.act)) {
                run(std::integral_constant<Form, kAnySigmoid>{});
            } else {
                run(std::integral_constant<Form, kAny>{});
            }
            // the next tile's first inputs, if this one had no steps to ask for them
            if (asked - n < min(kParts, next_all))
                ask(n, 0, 0, next_all, next_row, next_col);
        }
    }
};

// The tiles of a cluster, in order: a lane works out one of the next 32, a
// shuffle hands the next one to the warp (the divisions and the search for the
// group take longer than a block).
template <Mode kMode, int kRows, int kStep, int kParts>
struct TileWalk {
    Tile mine;
    int32_t idx, step, ntiles, mt, nt;
    int32_t n;

    __device__ __forceinline__ TileWalk(int32_t idx0, int32_t stride, int32_t rows, int32_t cols,
                                        int32_t total)
        : idx(idx0), step(stride), ntiles(total), mt(rows), nt(cols), n(0)
    {
    }
    // Whether there is another tile; next() then returns it.
    __device__ __forceinline__ bool more() const { return idx < ntiles; }
    __device__ __forceinline__ Tile next(const MmArgs &p, const int32_t *off, const int32_t *first)
    {
        if ((n & 31) == 0) {
            const int64_t at = idx + static_cast<int64_t>(threadIdx.x & 31) * step;
            mine = tile_at<kMode, kRows, kStep, kParts>(static_cast<int32_t>(min(at, static_cast<int64_t>(ntiles - 1))),
                                         p, off, first, mt, nt);
        }
        Tile t;
        const int src = n & 31;
        t.g = __shfl_sync(0xffffffffu, mine.g, src);
        t.row = __shfl_sync(0xffffffffu, mine.row, src);
        t.n0 = __shfl_sync(0xffffffffu, mine.n0, src);
        t.end = __shfl_sync(0xffffffffu, mine.end, src);
        t.blocks = __shfl_sync(0xffffffffu, mine.blocks, src);
        t.xblk = __shfl_sync(0xffffffffu, mine.xblk, src);
        t.arow = __shfl_sync(0xffffffffu, mine.arow, src);
        t.brow = __shfl_sync(0xffffffffu, mine.brow, src);
        n++;
        idx = idx > ntiles - step ? ntiles : idx + step;
        return t;
    }
};

// The same for a warp whose registers are needed: the next tiles lie in shared
// memory, kNotes at a time, and the rest is worked out from what is there.
template <Mode kMode, int kRows, int kStep, int kParts>
struct NoteWalk {
    int4 *notes;
    int32_t idx;
    uint32_t n;

    __device__ __forceinline__ Tile next(const MmArgs &p, const int32_t *off, const int32_t *first,
                                         int32_t step, int32_t ntiles)
    {
        if (n % kNotes == 0) {
            const int lane = threadIdx.x & 31;
            __syncwarp();
            if (lane < kNotes) {
                const int64_t at = idx + static_cast<int64_t>(lane) * step;
                const Tile t = tile_at<kMode, kRows, kStep, kParts>(
                    static_cast<int32_t>(min(at, static_cast<int64_t>(ntiles - 1))), p, off, first,
                    first[p.G + 1], (p.N + kStep - 1) / kStep);
                notes[lane] = make_int4(t.g, t.row, t.n0, t.end);
            }
            __syncwarp();
        }
        const int4 v = notes[n % kNotes];
        Tile t = {};
        t.g = v.x;
        t.row = v.y;
        t.n0 = v.z;
        t.end = v.w;
        t.blocks = v.x < p.G ? p.KB : 0;
        n++;
        idx = idx > ntiles - step ? ntiles : idx + step;
        return t;
    }
};

// The scales of one line (a row of c, a column or a weight tile) for up to
// kScaleBlocks consecutive blocks, `step` floats apart, from `s` on; `vec`: the
// four are one aligned vector.
__device__ __forceinline__ float4 load_scales(const float *s, int64_t step, int32_t n, bool vec)
{
    if (vec)
        return __ldg(reinterpret_cast<const float4 *>(s));
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (n > 0)
        v.x = __ldg(s);
    if (n > 1)
        v.y = __ldg(s + step);
    if (n > 2)
        v.z = __ldg(s + 2 * step);
    if (n > 3)
        v.w = __ldg(s + 3 * step);
    return v;
}

// Persistent: one CTA per SM, in clusters of kCtas.  Every CTA loads 128 rows of
// a and its share of the rows of b per block and owns 128 rows of the
// accumulator.  Warps 0-7 add up the scaled blocks (warp w: TMEM lanes 32 (w mod
// 4).., half w / 4 of the columns), warp 8 issues the tensor copies, warp 9 of
// the cluster's first CTA the MMAs, warp 10 fetches the scales of the columns
// where every column has its own.  Two TMEM buffers: the MMAs of block b + 1 run
// while block b is scaled and added.
//
// What bounds it.  A block of a 256 x 256 tile takes the tensor cores 512 cycles
// and its operands 64 KB of shared-memory traffic per SM (512 cycles as well), but
// the warps 0-7 about 820: the TMEM loads, 64 packed FMAs a thread (256 cycles for
// the two warps of a scheduler) and about 20 more instructions a warp at their full
// latency, which two warps a scheduler do not hide.  16384 x 4096 x 7168: 337 us
// (2.86 PFLOP/s) with the L2 flushed, 375 us back to back at the lower clocks that
// this draws; without scaling and adding the same loop takes 285 us.  With a scale
// per column it is twice the FMAs and a shared load per four columns: 540 us.
// Why so: pairs of CTAs halve the traffic of b (one CTA a tile: 415 us before the
// rest); 256 accumulator columns need 128 registers a thread, so the other roles
// give theirs up, down to 104 (at 56 they spill, and the kernel takes 10 to 20 %
// longer); 192-column tiles wait more often per column (410
// us); half-tile MMAs read a twice (500 us); 16 adding warps have too few registers
// (414 us and more).
template <int kCtas, Mode kMode, Out kOut, Epi kEpi>
__global__ void __launch_bounds__(kMmThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ MmMaps maps, const MmArgs p)
{
    constexpr bool kGatedTile = kEpi == kGated;
    using S = Shape<kCtas, kOut, kEpi>;
    constexpr int BN = S::bn, kCols = S::cols, kStages = S::stages;
    constexpr int kTmemCols = 2 * BN, kBufCols = BN;
    constexpr bool kColScale = kMode != kTileScale;
    constexpr int kCopyWarp = kPromoteWarps, kMmaWarp = kCopyWarp + 1, kColWarp = kMmaWarp + 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sA = smem, *sB = sA + kStages * S::a_bytes, *sC = sB + kStages * S::b_bytes;
    using Tail = MmTail<kCtas, kOut, kEpi>;
    Tail &t = *reinterpret_cast<Tail *>(sC + kPromoteWarps * S::warp_bytes);
    int32_t *off = reinterpret_cast<int32_t *>(&t + 1), *first = off + p.G + 2;

    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kCtas == 1 ? 0 : cluster_rank(), rank0 = rank;
    if (wid == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < kStages; i++) {
                mbar_init(&t.full[i], 1);
                mbar_init(&t.empty[i], 1);
            }
            for (int i = 0; i < 2; i++) {
                mbar_init(&t.acc_full[i], 1);
                mbar_init(&t.acc_empty[i], kCtas * kPromoteWarps);
                mbar_init(&t.scale_full[i], 1);
                mbar_init(&t.scale_empty[i], kPromoteWarps);
            }
            if (S::fetches)
                for (int i = 0; i < kPromoteWarps * S::slots; i++)
                    mbar_init(&t.in_full[0][0] + i, 1);
            t.abort = 0;
            mbar_init_fence();
        }
        __syncwarp();
        tmem_alloc<kCtas>(&t.tmem, kTmemCols);
    }
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    if (wid == 0) {
        const bool bad = load_row_groups(p.offs, p.G, p.M, kMode == kWgrad ? 128 : kCtas * kRowsM,
                                         off, first);
        if (bad && p.dev_status && blockIdx.x == 0 && lane == 0)
            atomicOr(p.dev_status, 1);
    }
    tc_fence_before();
    __syncthreads();
    if (kCtas > 1) {  // the barriers of both CTAs are set up
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    const uint32_t tmem = t.tmem;
    volatile int32_t *abort = &t.abort;
    const int32_t mt = kMode == kWgrad ? (p.R + kCtas * kRowsM - 1) / (kCtas * kRowsM)
                                       : first[p.G + 1];
    const int32_t nt = (p.N + S::step - 1) / S::step;
    const int32_t ntiles = mt * nt * (kMode == kWgrad ? p.G : 1);
    TileWalk<kMode, kCtas * kRowsM, S::step, kGatedTile ? 2 : 1> walk(blockIdx.x / kCtas, gridDim.x / kCtas, mt, nt, ntiles);

    if (wid >= kPromoteWarps) {
        regs_down<other_regs(kColScale)>();
        if (wid == kCopyWarp) {
            const uint32_t full0 = smem_u32(t.full), empty0 = smem_u32(t.empty);
            const uint32_t fill0 = kCtas == 1 ? full0 : cluster_addr(t.full, 0);
            const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
            uint32_t s = 0, ph = 1;
            while (!*abort && walk.more()) {
                const Tile tl = walk.next(p, off, first);
                const int32_t arow = tl.arow + rank * kRowsM;
                const int32_t brow = tl.brow + rank * (kGatedTile ? S::box_rows : S::b_rows);
                int32_t x = tl.xblk * kBlockK;
                for (int32_t b = 0; b < tl.blocks; b++, x += kBlockK) {
                    warp_wait(empty0 + 8 * s, ph, abort);
                    if (*abort)
                        break;
                    if (elect_one()) {
                        if (rank == 0)
                            mbar_arrive_expect_tx(&t.full[s], kCtas * (S::a_bytes + S::b_bytes));
                        if (kCtas == 1)
                            tma_load_2d(sA + s * S::a_bytes, &maps.a, x, arow, &t.full[s]);
                        else
                            tma_load_2d_pair(a0 + s * S::a_bytes, &maps.a, x, arow, fill0 + 8 * s);
                        // gated: gate rows, the up rows beside them, the next gate rows, ..
#pragma unroll
                        for (int i = 0; i < S::b_rows / S::box_rows; i++) {
                            const int32_t at = s * S::b_bytes + i * S::box_rows * kBlockK;
                            const int32_t row = brow + (i >> 1) * S::box_rows + (i & 1) * p.N;
                            if (kCtas == 1)
                                tma_load_2d(sB + at, &maps.b, x, row, &t.full[s]);
                            else
                                tma_load_2d_pair(b0 + at, &maps.b, x, row, fill0 + 8 * s);
                        }
                    }
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // every stage has been consumed: the last arrivals of the MMAs, which
            // come from the pair's first CTA, find this CTA's barriers
            for (int k = 0; k < kStages; k++) {
                warp_wait(empty0 + 8 * s, ph, abort);
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (*abort) {  // no copy may land after the CTA is gone: a millisecond is plenty
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000)
                    ;
            }
        } else if (wid == kMmaWarp && rank == 0) {
            constexpr uint32_t idesc = idesc_e4m3(kCtas * kRowsM, BN);
            const uint64_t da0 = smem_desc_sw128(sA), db0 = smem_desc_sw128(sB);
            const uint32_t full0 = smem_u32(t.full), empty0 = smem_u32(t.empty);
            const uint32_t acc_full0 = smem_u32(t.acc_full), acc_empty0 = smem_u32(t.acc_empty);
            uint32_t s = 0, ph = 0, it = 0;
            uint64_t da = da0, db = db0;
            while (!*abort && walk.more()) {
                const int32_t blocks = walk.next(p, off, first).blocks;
                for (int32_t b = 0; b < blocks; b++, it++) {
                    const uint32_t buf = it & 1;
                    warp_wait(full0 + 8 * s, ph, abort);
                    warp_wait(acc_empty0 + 8 * buf, ((it >> 1) & 1) ^ 1, abort);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kBlockK / 32; k++)
                            mma_e4m3<kCtas>(tmem + buf * kBufCols, da + 2 * k, db + 2 * k, idesc, k > 0);
                        mma_commit<kCtas>(acc_full0 + 8 * buf);
                        mma_commit<kCtas>(empty0 + 8 * s);
                    }
                    s++;
                    da += S::a_bytes >> 4;
                    db += S::b_bytes >> 4;
                    if (s == kStages) {
                        s = 0;
                        ph ^= 1;
                        da = da0;
                        db = db0;
                    }
                }
            }
            if (*abort) {  // no MMA may be in flight when TMEM is freed
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000)
                    ;
            }
        } else if (kColScale && wid == kColWarp) {
            constexpr int kPer = BN / 32;  // columns of a lane
            const bool vec = kMode == kRowScale && p.KB % 4 == 0;
            uint32_t gq = 0;
            while (!*abort && walk.more()) {
                const Tile tl = walk.next(p, off, first);
                for (int32_t b = 0; b < tl.blocks; b += kScaleBlocks, gq++) {
                    const uint32_t slot = gq & 1;
                    warp_wait(smem_u32(&t.scale_empty[slot]), ((gq >> 1) & 1) ^ 1, abort);
#pragma unroll
                    for (int i = 0; i < kPer; i += 2) {
                        float4 v[2];
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int at = lane + 32 * (i + h);
                            // gated: half, gate or up, column
                            const int32_t col =
                                min(tl.n0 + (kGatedTile ? at / 128 * 64 + at % 64 : at), p.N - 1);
                            const int64_t set = kGatedTile ? 2 * tl.g + at / 64 % 2 : tl.g;
                            const float *s =
                                kMode == kWgrad
                                    ? p.sb + static_cast<int64_t>(tl.xblk + b) * p.N + col
                                    : p.sb + (set * p.N + col) * p.KB + b;
                            v[h] = load_scales(s, kMode == kWgrad ? p.N : 1, tl.blocks - b, vec);
                        }
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            float *to = &t.col_scale[slot][0][lane + 32 * (i + h)];
                            to[0] = v[h].x;
                            to[BN] = v[h].y;
                            to[2 * BN] = v[h].z;
                            to[3 * BN] = v[h].w;
                        }
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&t.scale_full[slot]);
                }
            }
        }
        __syncwarp();
    } else {
        regs_up<promote_regs(kColScale)>();
        // What follows from the thread's number is worked out anew for every tile and for
        // its end where the kernel has an epilogue: kept, it would take registers that
        // the sums and the epilogue need (spills of the loop's own values were the price).
        constexpr bool kNoted = kEpi != kPlain;
        const bool aligned = static_cast<int64_t>(p.N) * (kOut == kF32 ? 4 : 2) % 16 == 0;
        uint32_t it = 0, gq = 0, nbox = 0;
        // The scales of the row and (kTileScale) of the weight tile that the columns
        // lie in, fetched two blocks ahead: those of a tile's first blocks before the
        // output of the tile before.
        const int64_t step = kMode == kWgrad ? p.R : 1;
        const float *sa = nullptr, *sb = nullptr;
        float a0 = 0.0f, a1 = 0.0f, b0 = 1.0f, b1 = 1.0f;
        // gated: the same for the up projection, whose weight tiles follow the gate's
        float u0 = 1.0f, u1 = 1.0f;
        const int64_t up_step = static_cast<int64_t>(p.sb_rows) * p.KB;
        constexpr bool kTwoScales = kGatedTile && !kColScale;
        auto open_tile = [&](const Tile &t) {
            const int tid = kNoted ? fresh_tid() : static_cast<int>(threadIdx.x);
            const int wid = tid >> 5, lane = tid & 31, half = wid >> 2;
            const uint32_t rank = kNoted && kCtas > 1 ? cluster_rank() : rank0;
            const int32_t row = t.row + rank * kRowsM + 32 * (wid & 3) + lane;
            if (kMode == kWgrad)
                sa = p.sa + static_cast<int64_t>(t.xblk) * p.R + min(row, p.R - 1);
            else
                sa = p.sa + static_cast<int64_t>(min(row, p.M - 1)) * p.KB;
            if (!kColScale)
                sb = p.sb + (static_cast<int64_t>(t.g) * (kGatedTile ? 2 : 1) * p.sb_rows +
                             min((t.n0 + (kGatedTile ? 0 : half * kCols)) / 128, p.sb_rows - 1)) *
                                p.KB;
            if (t.blocks > 0) {
                a0 = __ldg(sa);
                if (!kColScale)
                    b0 = __ldg(sb);
                if (kTwoScales)
                    u0 = __ldg(sb + up_step);
            }
            if (t.blocks > 1) {
                a1 = __ldg(sa + step);
                if (!kColScale)
                    b1 = __ldg(sb + 1);
                if (kTwoScales)
                    u1 = __ldg(sb + up_step + 1);
            }
            sa += 2 * step;
            sb += 2;
        };
        int32_t noted_idx = blockIdx.x / kCtas;
        uint32_t noted_n = 0;
        const auto another = [&] { return kNoted ? noted_idx < ntiles : walk.more(); };
        const auto take = [&] {
            if constexpr (kNoted) {
                NoteWalk<kMode, kCtas * kRowsM, S::step, kGatedTile ? 2 : 1> noted{
                    t.notes[fresh_tid() >> 5], noted_idx, noted_n};
                const Tile v = noted.next(p, off, first, gridDim.x / kCtas, ntiles);
                noted_idx = noted.idx;
                noted_n = noted.n;
                return v;
            } else {
                return walk.next(p, off, first);
            }
        };
        bool more = another();
        Tile next = {};
        if (more) {
            next = take();
            open_tile(next);
        }
        uint32_t asked = 0;
        if (S::fetches && more) {
            Finish<kCtas, kMode, kOut, kEpi> fin(p, maps, sC + wid * S::warp_bytes,
                                                 t.in_full[wid], t.bias[0], 0, 0);
            const int half = wid >> 2;
            const uint32_t rank = rank0;
            const int32_t row = next.row + rank * kRowsM + 32 * (wid & 3);
            const int32_t col = next.n0 + half * kCols;
            fin.ask(0, 0, 0, fin.boxes_of(row, next.end, col), row, col);
            asked = fin.asked;
        }
        // An exchange between warps needs both of them: they leave the loop by a
        // common vote (below) then.
        bool stop = false;
        uint32_t parity = 0;
        while (more && !(kOut == kE4m3 ? stop : *abort != 0)) {
            const Tile tl = next;
            const int32_t blocks = tl.blocks;
            uint64_t acc[kCols / 2];
#pragma unroll
            for (int e = 0; e < kCols / 2; e++)
                acc[e] = 0;
            {  // (what follows from tid is gone before the epilogue)
                const int tid = kNoted ? fresh_tid() : static_cast<int>(threadIdx.x);
                const int wid = tid >> 5, half = wid >> 2;
                const bool leader = (tid & 31) == 0;
                const uint32_t lane_base = (kNoted ? *static_cast<volatile uint32_t *>(&t.tmem) : tmem) +
                                           (static_cast<uint32_t>(32 * (wid & 3)) << 16) + half * kCols;
                const uint32_t acc_full0 = smem_u32(t.acc_full);
                const uint32_t read0 = kCtas == 1 ? smem_u32(t.acc_empty) : cluster_addr(t.acc_empty, 0);
                const uint32_t scale_full0 = smem_u32(t.scale_full);
                const uint32_t scale_empty0 = smem_u32(t.scale_empty);
                // A wait that gives up does not leave the loop (the other warps' waits
                // end soon as well); the flag is looked at behind it.
#pragma unroll 1
                for (int32_t b = 0; b < blocks; b++, it++) {
                    const float s = kColScale ? a0 : a0 * b0;
                    const float su = kTwoScales ? a0 * u0 : s;
                    a0 = a1;
                    b0 = b1;
                    if (kTwoScales)
                        u0 = u1;
                    if (b + 2 < blocks) {
                        a1 = __ldg(sa);
                        sa += step;
                        if (kTwoScales)
                            u1 = __ldg(sb + up_step);
                        if (!kColScale)
                            b1 = __ldg(sb++);
                    }
                    const uint32_t buf = it & 1, slot = gq & 1;
                    const float *cols = &t.col_scale[slot][b % kScaleBlocks][half * kCols];
                    if (kColScale && b % kScaleBlocks == 0)
                        warp_wait(scale_full0 + 8 * slot, (gq >> 1) & 1, abort);
                    warp_wait(acc_full0 + 8 * buf, (it >> 1) & 1, abort);
                    tc_fence_after();
                    const uint64_t sc = pack2(__float_as_uint(s), __float_as_uint(s));
                    const uint64_t scu = kTwoScales ? pack2(__float_as_uint(su), __float_as_uint(su)) : sc;
                    const uint32_t addr = lane_base + buf * kBufCols;
                    // kChunk columns at a time; with a scale per column, those of the
                    // chunk are fetched while it is on its way (16 columns: registers)
                    constexpr int kChunk = kColScale ? 16 : 32;
#pragma unroll
                    for (int c = 0; c < kCols / kChunk; c++) {
                        uint32_t r[kChunk];
                        uint4 cs[kColScale ? 4 : 1];
                        if (kColScale) {
                            tmem_ld16(addr + kChunk * c, r);
#pragma unroll
                            for (int q = 0; q < 4; q++)
                                cs[kColScale ? q : 0] =
                                    *reinterpret_cast<const uint4 *>(cols + kChunk * c + 4 * q);
                        } else {
                            tmem_ld32(addr + kChunk * c, r);
                        }
                        tmem_wait_ld();
                        if (c + 1 == kCols / kChunk) {  // the buffer has been read
                            tc_fence_before();
                            mbar_arrive_cluster(read0 + 8 * buf, leader);
                        }
                        uint64_t *o = acc + kChunk / 2 * c;
#pragma unroll
                        for (int e = 0; e < kChunk; e += 4) {
                            if (kColScale) {
                                const uint4 q = cs[kColScale ? e / 4 : 0];
                                mul_fma2(o[e / 2], r[e], r[e + 1], q.x, q.y, sc);
                                mul_fma2(o[e / 2 + 1], r[e + 2], r[e + 3], q.z, q.w, sc);
                            } else {
                                const uint64_t f = kTwoScales && kChunk * c >= kCols / 2 ? scu : sc;
                                fma2(o[e / 2], r[e], r[e + 1], f);
                                fma2(o[e / 2 + 1], r[e + 2], r[e + 3], f);
                            }
                        }
                    }
                    if (kColScale && (b % kScaleBlocks == kScaleBlocks - 1 || b + 1 == blocks)) {
                        __syncwarp();
                        mbar_arrive_cluster(scale_empty0 + 8 * slot, leader);
                        gq++;
                    }
                }
            }
            more = another();
            if (more) {
                next = take();
                open_tile(next);
            }
            const int tid = kNoted ? fresh_tid() : static_cast<int>(threadIdx.x);
            const int wid = tid >> 5, lane = tid & 31, half = wid >> 2;
            const uint32_t rank = kNoted && kCtas > 1 ? cluster_rank() : rank0;
            const int32_t col0 = tl.n0 + half * (kGatedTile ? kCols / 2 : kCols);
            const int32_t row0 = tl.row + rank * kRowsM + 32 * (wid & 3);
            uint8_t *stage = sC + wid * S::warp_bytes;
            if constexpr (kEpi == kAct) {
                // 128 columns' bias: a lane fetches every 32nd
                if (p.e.bias) {
#pragma unroll
                    for (int i = 0; i < kCols / 32; i++) {
                        const int32_t col = col0 + 32 * i + lane;
                        t.bias[wid][32 * i + lane] =
                            tl.g < p.G && col < p.N
                                ? __ldg(p.e.bias + static_cast<int64_t>(tl.g) * p.N + col)
                                : 0.0f;
                    }
                    __syncwarp();
                }
            }
            if constexpr (kEpi == kPlain) {
                const bool ok = __all_sync(0xffffffffu, *abort == 0);
                const int32_t rows = min(32, tl.end - row0);
                if (ok && rows > 0) {
                    const int64_t out0 = (kMode == kWgrad ? static_cast<int64_t>(tl.g) * p.R : 0) + row0;
                    const bool add = kMode == kWgrad && p.add;
                    const bool bulk = aligned && rows == 32 && !add;
                    if (kOut != kF32 && add && lane < rows)
                        add_bf16<kCols>(p.c, (out0 + lane) * p.N, col0, p.N, acc);
#pragma unroll
                    for (int x = 0; x < kCols / kBoxCols; x++) {
                        const int32_t col = col0 + kBoxCols * x;
                        if (col >= p.N)
                            continue;
                        // the box used S::boxes boxes ago has been read
                        uint8_t *box = stage + nbox % S::boxes * S::box_bytes;
                        nbox++;
                        if (lane == 0)
                            tma_store_wait_read<S::boxes - 1>();
                        __syncwarp();
                        stage_box<kOut == kF32>(box, acc + kBoxCols / 2 * x);
                        fence_async_shared();
                        __syncwarp();
                        if (!bulk) {
                            if (add)
                                store_box<kOut == kF32, true>(p.c, box, out0, rows, col, p.N, p.N);
                            else
                                store_box<kOut == kF32, false>(p.c, box, out0, rows, col, p.N, p.N);
                            __syncwarp();
                        }
                        if (lane == 0) {
                            if (bulk)
                                tma_store_2d(&maps.c, box, col, static_cast<int32_t>(out0));
                            tma_store_commit();  // a group for every box
                        }
                    }
                }
            } else {
                Finish<kCtas, kMode, kOut, kEpi> fin(p, maps, stage, t.in_full[wid],
                                                     t.bias[kEpi == kAct ? wid : 0], nbox, asked);
                fin.begin(row0, tl.end, tl.g, col0, kGatedTile ? kCols / 2 : kCols);
                if constexpr (kOut == kE4m3) {
                    uint32_t(*row_max)[kRowsM] = t.row_max[parity];
                    parity ^= 1;
                    const uint32_t most = fin.gated(acc, col0);
                    const int r = 32 * (wid & 3) + lane;
                    row_max[half][r] = most;
                    stop = named_barrier_or(1 + (wid & 3), 64, *abort != 0);
                    if (!stop)
                        fin.quantized(acc, col0, max(most, row_max[half ^ 1][r]));
                } else if (__all_sync(0xffffffffu, *abort == 0)) {
                    fin.store(acc, col0, next.row + rank * kRowsM + 32 * (wid & 3),
                              more ? next.end : 0, next.n0 + half * kCols, abort);
                }
                nbox = fin.n;
                asked = fin.asked;
            }
        }
        if (kEpi == kPlain ? lane == 0 : elect_one())
            tma_store_wait();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (kCtas > 1) {  // nothing of the pair reaches into this CTA any more
        cluster_arrive();
        cluster_wait();
    }
    if (wid == kMmaWarp)
        tmem_free<kCtas>(tmem, kTmemCols);
    if (threadIdx.x == 0 && t.abort && p.dev_status)
        atomicOr(p.dev_status, 2);
}

// Both operands: [rows, K bytes] matrices cut into 128-byte blocks along K.
template <int kCtas, Mode kMode, Out kOut, Epi kEpi>
fq_status launch_matmul(const uint8_t *a, int64_t a_rows, const uint8_t *b, int64_t b_rows,
                        int64_t K, int64_t c_rows, const MmArgs &p, cudaStream_t st)
{
    using S = Shape<kCtas, kOut, kEpi>;
    MmMaps maps = {};
    // a matrix of `pitch` elements a row, written (or read) in boxes of 32 rows and kBoxCols
    // columns (64 bytes of codes); rows that are not 16-byte aligned are not written so
    auto out_map = [&](CUtensorMap *map, const void *c, int64_t pitch, Out type) {
        const int64_t size = type == kF32 ? 4 : (type == kBf16 ? 2 : 1);
        return pitch * size % 16 != 0 ||
               encode_tensor_map_2d(map, type == kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : type == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                                    c, pitch, c_rows, static_cast<uint64_t>(pitch) * size,
                                    type == kE4m3 ? 64 : kBoxCols, 32,
                                    type == kF32 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                 : CU_TENSOR_MAP_SWIZZLE_64B,
                                    false);
    };
    const int64_t N = p.N, wide = kEpi == kGatedGrad ? 2 * N : N;
    bool ok = encode_tensor_map_2d(&maps.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, a_rows, K,
                                   kBlockK, kRowsM, CU_TENSOR_MAP_SWIZZLE_128B, true) &&
              encode_tensor_map_2d(&maps.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, K, b_rows, K,
                                   kBlockK, S::box_rows, CU_TENSOR_MAP_SWIZZLE_128B, true) &&
              out_map(&maps.c, p.c, wide, kOut);
    if (p.e.side)
        ok = ok && out_map(&maps.d, p.e.side, kEpi == kGated ? 2 * N : N, kBf16);
    if (S::fetches && p.e.in)
        ok = ok && out_map(&maps.in, p.e.in, wide, kOut);
    if (!ok) {
        set_last_cuda_error(static_cast<int>(cudaErrorNotSupported));
        return FQ_ERR_CUDA;
    }
    const auto kern = fp8_matmul_kernel<kCtas, kMode, kOut, kEpi>;
    const size_t dyn = 1024 + S::stages * (S::a_bytes + S::b_bytes) +
                       kPromoteWarps * S::warp_bytes +
                       sizeof(MmTail<kCtas, kOut, kEpi>) + 2 * (p.G + 2) * sizeof(int32_t);
    static_assert(1024 + S::stages * (S::a_bytes + S::b_bytes) +
                          kPromoteWarps * S::warp_bytes +
                          sizeof(MmTail<kCtas, kOut, kEpi>) +
                          2 * (FQ_COLS_MAX_GROUPS + 2) * sizeof(int32_t) <=
                      227 * 1024,
                  "shared memory of a CTA");
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(dyn)) != cudaSuccess)
        return launch_status();
    const int64_t rows = kCtas * kRowsM, nt = (p.N + S::step - 1) / S::step;
    const int64_t tiles = kMode == kWgrad ? (p.R + rows - 1) / rows * nt * p.G
                                          : ((p.M + rows - 1) / rows + p.G + 1) * nt;
    const int64_t most = sm_count() / kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kCtas * (tiles < most ? tiles : most)));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, maps, p) != cudaSuccess)
        return launch_status();
    return launch_status();
}

// ---------------------------------------------------------------- few rows

// The product for few rows per group (a decode step): the weights are read once
// and bound the time, so the roles are swapped.  The 128 rows of the MMA are
// weight rows (columns of c), its columns kT rows of a, and what is in flight is
// weights: 2 CTAs per SM with 4 to 6 stages of 16 KB of them (3 CTAs with 4 stages
// were 8 % slower, 1 CTA with 11 stages 5 %).  A lane of the
// accumulator is a column of c; a block's products are scaled by the row's scale,
// which a shuffle hands round.  With few tiles the blocks of K are split over a
// cluster of S CTAs, whose sums are added through shared memory in rank order.
// Bound by HBM: 512 rows over 32 experts of 4096 x 7168 in 152 to 163 us, 5.8 to 6.2
// TB/s; one row through 14336 x 4096 in 15.6 us, 3.8 TB/s, of which the launch, the
// set-up and the first and last bytes' latency are about 6 us.
// Gated: a stage holds 128 gate rows and the up rows beside them, a lane both sums.
// Two CTAs share an SM up to 480 groups, whose offsets lie behind the stages (a quantized
// gated result by tiles of 32 rows: 371, for the magnitudes beside them; up to 1024 with the
// tiles of 32 and 64 rows that are not gated, or of 16 gated).  Above, one does: 4 rows in
// each of 464 groups of 512 x 2048 84 us with two, 88 with one; with 512 groups a stage fewer
// for two instead of one took 94.2 for 93.7, 12 rows in each 100.4 for 98.4, and gated by
// tiles of 32 rows 187 for 194.
template <int kT, bool kGatedTile>
struct Few {
    // CTAs per SM and their stages: about 200 KB of weights in flight per SM
    static constexpr int per_sm = 2;
    static constexpr int parts = kGatedTile ? 2 : 1;
    static constexpr int stages = kGatedTile ? 3 : (kT == 16 ? 6 : (kT == 32 ? 5 : 4));
    static constexpr int w_bytes = parts * 128 * kBlockK, x_bytes = kT * kBlockK;
    static constexpr int tmem_cols = 128, buf_cols = parts * kT, bufs = tmem_cols / buf_cols;
    static constexpr int threads = 6 * 32;
};

// Largest magnitudes of a block: of every row of a by every warp.
template <int kT, bool kQuantized>
struct FewMax {
    uint32_t row_max[2][4][kT];
};
template <int kT>
struct FewMax<kT, false> {};

template <int kT, bool kGatedTile, bool kQuantized>
struct FewTail : FewMax<kT, kQuantized> {
    using F = Few<kT, kGatedTile>;
    uint64_t full[F::stages], empty[F::stages];
    uint64_t acc_full[F::bufs], acc_empty[F::bufs];
    uint32_t tmem;
    int32_t abort;
    // int32 off[G + 2], first[G + 2] follow
};

// Bytes of shared memory that a CTA is launched with; two CTAs share an SM with 113 KB each.
template <int kT, bool kGatedTile, bool kQuantized>
constexpr int few_bytes(int32_t G)
{
    using F = Few<kT, kGatedTile>;
    return 1024 + F::stages * (F::w_bytes + F::x_bytes) +
           static_cast<int>(sizeof(FewTail<kT, kGatedTile, kQuantized>)) +
           2 * (G + 2) * static_cast<int>(sizeof(int32_t));
}

// The end of a tile of few rows: what a lane makes of the sums of column n, two rows at a
// time (the second of them may be missing).  The form of the activation is chosen once a
// tile: with a branch a row, 8192 x 512 x 2048 in 256 groups took 97 us with bias, silu,
// residual and z where two rows at a time take 87, and 63 with what is read (residual, z)
// asked for before the first block.
template <Out kOut, Epi kEpi>
struct FewFinish {
    static constexpr bool kWideOut = kOut == kF32;
    const MmArgs &p;
    int g;
    int32_t n;
    const Act act;

    template <bool kWide>
    static __device__ __forceinline__ void put(void *c, int64_t at, int64_t pitch, bool two, uint64_t v)
    {
        float f[2];
        unpack2(v, f[0], f[1]);
        if (kWide) {
            float *to = static_cast<float *>(c) + at;
            to[0] = f[0];
            if (two)
                to[pitch] = f[1];
        } else {
            uint16_t *to = static_cast<uint16_t *>(c) + at;
            const uint32_t w = cvt_bf16x2(f[0], f[1]);
            to[0] = static_cast<uint16_t>(w);
            if (two)
                to[pitch] = static_cast<uint16_t>(w >> 16);
        }
    }
    __device__ __forceinline__ float bias() const
    {
        return kEpi == kAct && p.e.bias && g < p.G
                   ? __ldg(p.e.bias + static_cast<int64_t>(g) * p.N + n)
                   : 0.0f;
    }
    // Whether there is something to read: not in rows of no group, whose gradients are 0
    // with z = 0.
    __device__ __forceinline__ bool reads() const
    {
        return kEpi == kAct ? p.e.in != nullptr : kEpi != kGated && g < p.G;
    }
    // What is read at row m: the residual, z, or gate and up (part), as it is stored and
    // as a number.
    __device__ __forceinline__ uint32_t fetch(int32_t m, int part) const
    {
        const int64_t at = (kEpi == kGatedGrad ? 2 * static_cast<int64_t>(m) + part : m) *
                               static_cast<int64_t>(p.N) + n;
        return kEpi == kAct && kWideOut ? static_cast<const uint32_t *>(p.e.in)[at]
                                        : static_cast<const uint16_t *>(p.e.in)[at];
    }
    static __device__ __forceinline__ float number(uint32_t v)
    {
        return kEpi == kAct && kWideOut ? __uint_as_float(v) : bf16_lo(v);
    }
    // The gated results of both sums, which go out too if they are asked for.
    template <bool kSigmoid>
    __device__ __forceinline__ uint64_t gated(int32_t m, bool two, uint64_t gate, uint64_t up) const
    {
        if (p.e.side) {
            const int64_t at = 2 * static_cast<int64_t>(m) * p.N + n, pitch = 2 * static_cast<int64_t>(p.N);
            put<false>(p.e.side, at, pitch, two, gate);
            put<false>(p.e.side, at + p.N, pitch, two, up);
        }
        return mul_x2(act.template value<kSigmoid>(gate), up);
    }
    // h as E4M3 by the factor r of its block (a NaN's: there is an infinity or a NaN in it).
    __device__ __forceinline__ void quantized(int32_t m, float h, float r) const
    {
        static_cast<uint8_t *>(p.c)[static_cast<int64_t>(m) * p.N + n] =
            r != r ? 0x7F : static_cast<uint8_t>(cvt_e4m3x2(h * r, 0.0f));
    }
    // v, v2: the sums; x, y: what was read; b: the bias
    template <bool kSigmoid>
    __device__ __forceinline__ void store(int32_t m, bool two, uint64_t v, uint64_t v2, uint64_t x,
                                          uint64_t y, float b) const
    {
        const int64_t at = static_cast<int64_t>(m) * p.N + n;
        if constexpr (kEpi == kAct) {
            v = add_x2(v, Act::both(b));
            if (p.e.side)
                put<false>(p.e.side, at, p.N, two, v);
            put<kWideOut>(p.c, at, p.N, two, add_x2(act.template value<kSigmoid>(v), x));
        } else if constexpr (kEpi == kGated) {
            put<kWideOut>(p.c, at, p.N, two, gated<kSigmoid>(m, two, v, v2));
        } else {
            uint64_t slope, value = act.template gradient<kSigmoid>(x, slope);
            if constexpr (kEpi == kGatedGrad) {
                const int64_t pitch = 2 * static_cast<int64_t>(p.N), to = at + static_cast<int64_t>(m) * p.N;
                put<kWideOut>(p.c, to, pitch, two, mul_x2(v, mul_x2(y, slope)));
                put<kWideOut>(p.c, to + p.N, pitch, two, mul_x2(v, value));
                value = mul_x2(value, y);
            } else {
                put<kWideOut>(p.c, at, p.N, two, mul_x2(v, slope));
            }
            if (p.e.side)
                put<false>(p.e.side, at, p.N, two, value);
        }
    }
};

// Warps 0-3 add up the blocks, warp 4 issues the tensor copies, warp 5 the MMAs.
template <int kT, Mode kMode, Out kOut, Epi kEpi>
__global__ void __launch_bounds__(Few<kT, kEpi == kGated>::threads, Few<kT, kEpi == kGated>::per_sm)
    fp8_matmul_few_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw,
                          const MmArgs p, const int32_t S)
{
    constexpr bool kGatedTile = kEpi == kGated;
    using F = Few<kT, kGatedTile>;
    constexpr int kParts = F::parts;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sW = smem, *sX = sW + F::stages * F::w_bytes;
    using Tail = FewTail<kT, kGatedTile, kOut == kE4m3>;
    Tail &t = *reinterpret_cast<Tail *>(sX + F::stages * F::x_bytes);
    int32_t *off = reinterpret_cast<int32_t *>(&t + 1), *first = off + p.G + 2;
    volatile int32_t *abort = &t.abort;
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t rank = S > 1 ? static_cast<int32_t>(cluster_rank()) : 0;

    if (wid == 5) {
        if (lane == 0) {
            for (int i = 0; i < F::stages; i++) {
                mbar_init(&t.full[i], 1);
                mbar_init(&t.empty[i], 1);
            }
            for (int i = 0; i < F::bufs; i++) {
                mbar_init(&t.acc_full[i], 1);
                mbar_init(&t.acc_empty[i], 4);
            }
            t.abort = 0;
            mbar_init_fence();
        }
        __syncwarp();
        tmem_alloc<1>(&t.tmem, F::tmem_cols);
    }
    griddep_wait();  // the previous kernel's outputs (PDL launch)
    griddep_launch_dependents();  // the next kernel may start its set-up
    if (wid == 0) {
        const bool bad = load_row_groups(p.offs, p.G, p.M, kT, off, first);
        if (bad && p.dev_status && blockIdx.x == 0 && lane == 0)
            atomicOr(p.dev_status, 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = t.tmem;
    // row tiles of all groups run fastest: tiles in flight share weights
    const int32_t mt = first[p.G + 1], nt = (p.N + 127) / 128, ntiles = mt * nt;
    const int32_t b_lo = static_cast<int32_t>(static_cast<int64_t>(p.KB) * rank / S);
    const int32_t b_hi = static_cast<int32_t>(static_cast<int64_t>(p.KB) * (rank + 1) / S);
    const int32_t idx0 = blockIdx.x / S, step = gridDim.x / S;

    if (wid == 4) {
        uint32_t s = 0, ph = 1;
        for (int32_t idx = idx0; idx < ntiles && !*abort; idx += step) {
            const int32_t j = idx / mt, i = idx - j * mt;
            const int g = group_of_tile(first, p.G + 1, i);
            if (g == p.G)
                continue;
            const int32_t row = off[g] + (i - first[g]) * kT, wrow = g * kParts * p.N + j * 128;
            for (int32_t b = b_lo; b < b_hi; b++) {
                warp_wait(smem_u32(&t.empty[s]), ph, abort);
                if (*abort)
                    break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&t.full[s], F::w_bytes + F::x_bytes);
#pragma unroll
                    for (int q = 0; q < kParts; q++)
                        tma_load_2d(sW + s * F::w_bytes + q * 128 * kBlockK, &tw, b * kBlockK,
                                    wrow + q * p.N, &t.full[s]);
                    tma_load_2d(sX + s * F::x_bytes, &tx, b * kBlockK, row, &t.full[s]);
                }
                if (++s == F::stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (*abort) {  // no copy may land after the CTA is gone: a millisecond is plenty
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000)
                ;
        }
    } else if (wid == 5) {
        constexpr uint32_t idesc = idesc_e4m3(128, kT);
        const uint64_t dw0 = smem_desc_sw128(sW), dx0 = smem_desc_sw128(sX);
        uint32_t s = 0, ph = 0, it = 0;
        for (int32_t idx = idx0; idx < ntiles && !*abort; idx += step) {
            if (group_of_tile(first, p.G + 1, idx % mt) == p.G)
                continue;
            for (int32_t b = b_lo; b < b_hi; b++, it++) {
                const uint32_t buf = it % F::bufs, bph = (it / F::bufs) & 1;
                warp_wait(smem_u32(&t.full[s]), ph, abort);
                warp_wait(smem_u32(&t.acc_empty[buf]), bph ^ 1, abort);
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t dw = dw0 + s * (F::w_bytes >> 4), dx = dx0 + s * (F::x_bytes >> 4);
#pragma unroll
                    for (int q = 0; q < kParts; q++)
#pragma unroll
                        for (int k = 0; k < kBlockK / 32; k++)
                            mma_e4m3<1>(tmem + buf * F::buf_cols + q * kT,
                                        dw + q * (128 * kBlockK >> 4) + 2 * k, dx + 2 * k, idesc,
                                        k > 0);
                    mma_commit<1>(smem_u32(&t.acc_full[buf]));
                    mma_commit<1>(smem_u32(&t.empty[s]));
                }
                if (++s == F::stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (*abort) {  // no MMA may be in flight when TMEM is freed
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000)
                ;
        }
    } else {
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * wid) << 16);
        constexpr int kHold = (kT + 31) / 32;  // rows' scales of a lane
        // a weight row's scale differs from the other lanes' or the other part's
        constexpr bool kOwnScale = kMode == kRowScale || kGatedTile;
        uint32_t it = 0, parity = 0;
        // the warps exchange magnitudes where c is quantized: they leave together
        bool stop = false;
        for (int32_t idx = idx0; idx < ntiles && !(kOut == kE4m3 ? stop : *abort != 0); idx += step) {
            const int32_t j = idx / mt, i = idx - j * mt;
            const int g = group_of_tile(first, p.G + 1, i);
            const int32_t row0 = off[g] + (i - first[g]) * kT;
            const int32_t rows = min(kT, off[g + 1] - row0);
            const int32_t n = j * 128 + 32 * wid + lane;
            const FewFinish<kOut, kEpi> fin{p, g, n, Act(p.e.act)};
            // What the epilogue reads is asked for some rows at a time, all of it before
            // the first block where it fits into registers.
            constexpr bool kReads = kEpi != kPlain && kEpi != kGated;
            constexpr int kIn = kEpi == kGatedGrad ? 2 : 1;
            constexpr int kSome = kIn * kT > 32 ? 32 / kIn : kT;
            uint32_t in[kReads ? kIn : 1][kReads ? kSome : 1] = {};
            const auto ask = [&](int e0) {
                if (kReads && n < p.N && fin.reads())
#pragma unroll
                    for (int q = 0; q < kIn; q++)
#pragma unroll
                        for (int e = 0; e < kSome; e++)
                            in[kReads ? q : 0][kReads ? e : 0] =
                                fin.fetch(row0 + min(e0 + e * S, rows - 1), q);
            };
            ask(rank);
            const float bias = n < p.N ? fin.bias() : 0.0f;
            float acc[kParts][kT];
#pragma unroll
            for (int q = 0; q < kParts; q++)
#pragma unroll
                for (int e = 0; e < kT; e++)
                    acc[q][e] = 0.0f;
            if (g < p.G) {
                const float *sa[kHold];
                float a[kHold], an[kHold];
#pragma unroll
                for (int h = 0; h < kHold; h++) {
                    sa[h] = p.sa + static_cast<int64_t>(
                                       min(row0 + min(lane + 32 * h, kT - 1), p.M - 1)) * p.KB;
                    a[h] = b_lo < b_hi ? __ldg(sa[h] + b_lo) : 0.0f;
                    an[h] = b_lo + 1 < b_hi ? __ldg(sa[h] + b_lo + 1) : 0.0f;
                }
                const float *sb = p.sb + (static_cast<int64_t>(g) * kParts * p.sb_rows +
                                          (kMode == kRowScale ? min(n, p.N - 1) : j)) * p.KB;
                const int64_t up = static_cast<int64_t>(p.sb_rows) * p.KB;
                float w[kParts], wn[kParts];
#pragma unroll
                for (int q = 0; q < kParts; q++) {
                    w[q] = b_lo < b_hi ? __ldg(sb + q * up + b_lo) : 0.0f;
                    wn[q] = b_lo + 1 < b_hi ? __ldg(sb + q * up + b_lo + 1) : 0.0f;
                }
                for (int32_t b = b_lo; b < b_hi; b++, it++) {
                    const uint32_t buf = it % F::bufs, bph = (it / F::bufs) & 1;
                    float sc[kHold], wk[kParts];
#pragma unroll
                    for (int h = 0; h < kHold; h++) {
                        sc[h] = kOwnScale ? a[h] : a[h] * w[0];
                        a[h] = an[h];
                        if (b + 2 < b_hi)
                            an[h] = __ldg(sa[h] + b + 2);
                    }
#pragma unroll
                    for (int q = 0; q < kParts; q++) {
                        wk[q] = w[q];
                        w[q] = wn[q];
                        if (b + 2 < b_hi)
                            wn[q] = __ldg(sb + q * up + b + 2);
                    }
                    warp_wait(smem_u32(&t.acc_full[buf]), bph, abort);
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < F::buf_cols / 16; c++) {
                        uint32_t r[16];
                        tmem_ld16(lanes + buf * F::buf_cols + 16 * c, r);
                        tmem_wait_ld16(r);
                        if (c + 1 == F::buf_cols / 16) {  // the buffer has been read
                            tc_fence_before();
                            mbar_arrive_cluster(smem_u32(&t.acc_empty[buf]), lane == 0);
                        }
#pragma unroll
                        for (int e = 0; e < 16; e++) {
                            const int q = 16 * c / kT, col = 16 * c % kT + e;
                            float v = __uint_as_float(r[e]);
                            if (kOwnScale)
                                v *= wk[q];
                            acc[q][col] = __fmaf_rn(
                                v, __shfl_sync(0xffffffffu, sc[col / 32], col % 32), acc[q][col]);
                        }
                    }
                }
            }
            if (S == 1) {
                if constexpr (kOut == kE4m3) {
                    static_assert(kT <= 32, "a lane for every row's scale");
                    float h[kT];
                    uint32_t(*row_max)[kT] = t.row_max[parity];
                    parity ^= 1;
                    const auto finish = [&](auto form) {
#pragma unroll
                        for (int e = 0; e < kT; e += 2) {
                            h[e] = h[e + 1] = 0.0f;
                            if (e < rows)
                                unpack2(fin.template gated<decltype(form)::value>(
                                            row0 + e, e + 1 < rows, pack2f(acc[0][e], acc[0][e + 1]),
                                            pack2f(acc[kParts - 1][e], acc[kParts - 1][e + 1])),
                                        h[e], h[e + 1]);
                        }
                    };
                    if (Act::sigmoid(p.e.act))
                        finish(std::true_type{});
                    else
                        finish(std::false_type{});
#pragma unroll
                    for (int e = 0; e < kT; e++) {
                        const uint32_t most =
                            __reduce_max_sync(0xffffffffu, __float_as_uint(h[e]) & 0x7FFFFFFFu);
                        if (lane == 0)
                            row_max[wid][e] = most;
                    }
                    stop = named_barrier_or(1, 128, *abort != 0);
                    // a lane works out a row's scale
                    float r, scale;
                    const int own = lane % kT;
                    e4m3_factors(max(max(row_max[0][own], row_max[1][own]),
                                     max(row_max[2][own], row_max[3][own])),
                                 r, scale);
                    if (wid == 0 && lane < rows && !stop)
                        p.e.scales[static_cast<int64_t>(row0 + lane) * (p.N / 128) + j] = scale;
#pragma unroll
                    for (int e = 0; e < kT; e++) {
                        const float by = __shfl_sync(0xffffffffu, r, e);
                        if (e < rows && !stop)
                            fin.quantized(row0 + e, h[e], by);
                    }
                } else if (n < p.N && *abort == 0) {
                    if constexpr (kEpi == kPlain) {
#pragma unroll
                        for (int e = 0; e < kT; e++) {
                            const int64_t at = static_cast<int64_t>(row0 + e) * p.N + n;
                            if (e < rows && kOut == kF32)
                                static_cast<float *>(p.c)[at] = acc[0][e];
                            if (e < rows && kOut != kF32)
                                static_cast<uint16_t *>(p.c)[at] =
                                    static_cast<uint16_t>(cvt_bf16x2(acc[0][e], 0.0f));
                        }
                    } else {
                        const auto read = [&](int q, int i) {
                            return kReads ? pack2f(fin.number(in[kReads ? q : 0][kReads ? i : 0]),
                                                   fin.number(in[kReads ? q : 0][kReads ? i + 1 : 0]))
                                          : Act::both(0.0f);
                        };
                        const auto finish = [&](auto form) {
#pragma unroll
                            for (int e0 = 0; e0 < kT; e0 += kSome) {
                                if (e0 > 0)
                                    ask(e0);
#pragma unroll
                                for (int i = 0; i < kSome; i += 2) {
                                    const int e = e0 + i;
                                    if (e < rows)
                                        fin.template store<decltype(form)::value>(
                                            row0 + e, e + 1 < rows, pack2f(acc[0][e], acc[0][e + 1]),
                                            pack2f(acc[kParts - 1][e], acc[kParts - 1][e + 1]),
                                            read(0, i), read(kIn - 1, i), bias);
                                }
                            }
                        };
                        if (Act::sigmoid(p.e.act))
                            finish(std::true_type{});
                        else
                            finish(std::false_type{});
                    }
                }
            } else {  // one tile: its stages are free, every copy has been waited for
                float *part = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int q = 0; q < kParts; q++)
#pragma unroll
                    for (int e = 0; e < kT; e++)
                        part[(q * kT + e) * 128 + 32 * wid + lane] = acc[q][e];
                // what has been read waits behind them, a thread's own
                if (kReads)
#pragma unroll
                    for (int q = 0; q < kIn; q++)
#pragma unroll
                        for (int e = 0; e < kSome; e++)
                            part[(kParts * kT + q * kSome + e) * 128 + 32 * wid + lane] =
                                fin.number(in[kReads ? q : 0][kReads ? e : 0]);
            }
        }
    }
    if (S > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        // CTA r adds up rows r, r + S, .. of the tile
        bool run = wid < 4 && idx0 < ntiles && *abort == 0;
        if (kOut == kE4m3 && wid < 4)
            run = !named_barrier_or(1, 128, !run);
        if (run) {
            const int32_t j = idx0 / mt, i = idx0 - j * mt;
            const int g = group_of_tile(first, p.G + 1, i);
            const int32_t row0 = off[g] + (i - first[g]) * kT;
            const int32_t rows = min(kT, off[g + 1] - row0);
            const int32_t n = j * 128 + 32 * wid + lane;
            const FewFinish<kOut, kEpi> fin{p, g, n, Act(p.e.act)};
            const float bias = n < p.N ? fin.bias() : 0.0f;
            uint32_t parity = 0;
            constexpr bool kReads = kEpi != kPlain && kEpi != kGated;
            constexpr int kIn = kEpi == kGatedGrad ? 2 : 1;
            constexpr int kSome = kIn * kT > 32 ? 32 / kIn : kT;
            const float *part = reinterpret_cast<const float *>(smem) + 32 * wid + lane;
            const auto finish = [&](auto form) {
                constexpr bool kSigmoid = decltype(form)::value;
                int i = 0;  // of this CTA's rows
                for (int32_t e = rank; e < rows; e += S, i++) {
                    float v[kParts], in[2] = {0.0f, 0.0f};
                    if constexpr (kReads) {
#pragma unroll
                        for (int q = 0; q < kIn; q++)
                            in[q] = i < kSome ? part[(kParts * kT + q * kSome + i) * 128]
                                    : n < p.N && fin.reads() ? fin.number(fin.fetch(row0 + e, q))
                                                             : 0.0f;
                    }
#pragma unroll
                    for (int q = 0; q < kParts; q++) {
                        float of[8];  // on their way at once
#pragma unroll
                        for (int r = 0; r < 8; r++)
                            of[r] = r < S ? ld_cluster_f32(cluster_addr(part + (q * kT + e) * 128, r))
                                          : 0.0f;
                        v[q] = 0.0f;
#pragma unroll
                        for (int r = 0; r < 8; r++)
                            if (r < S)
                                v[q] += of[r];
                    }
                    if constexpr (kOut == kE4m3) {
                        float h, none, r, scale;
                        unpack2(fin.template gated<kSigmoid>(row0 + e, false, Act::both(v[0]),
                                                             Act::both(v[kParts - 1])),
                                h, none);
                        const uint32_t most =
                            __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7FFFFFFFu);
                        uint32_t(*row_max)[kT] = t.row_max[parity];
                        parity ^= 1;
                        if (lane == 0)
                            row_max[wid][0] = most;
                        named_barrier_or(1, 128, false);
                        e4m3_factors(max(max(row_max[0][0], row_max[1][0]),
                                         max(row_max[2][0], row_max[3][0])),
                                     r, scale);
                        if (wid == 0 && lane == 0)
                            p.e.scales[static_cast<int64_t>(row0 + e) * (p.N / 128) + j] = scale;
                        fin.quantized(row0 + e, h, r);
                    } else if (n < p.N) {
                        if constexpr (kEpi == kPlain) {
                            const int64_t at = static_cast<int64_t>(row0 + e) * p.N + n;
                            if (kOut == kF32)
                                static_cast<float *>(p.c)[at] = v[0];
                            else
                                static_cast<uint16_t *>(p.c)[at] =
                                    static_cast<uint16_t>(cvt_bf16x2(v[0], 0.0f));
                        } else {
                            fin.template store<kSigmoid>(row0 + e, false, Act::both(v[0]),
                                                         Act::both(v[kParts - 1]), Act::both(in[0]),
                                                         Act::both(in[1]), bias);
                        }
                    }
                }
            };
            if (kEpi != kPlain && Act::sigmoid(p.e.act))
                finish(std::true_type{});
            else
                finish(std::false_type{});
        }
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (wid == 5)
        tmem_free<1>(tmem, F::tmem_cols);
    if (threadIdx.x == 0 && t.abort && p.dev_status)
        atomicOr(p.dev_status, 2);
}

// The CTAs that share a tile's blocks of K.  They are split while an SM has no more
// than one CTA (with 64 rows, which keep a CTA longer, two): 112 tiles of 14336 x 4096
// took 15 to 16 us for 1 to 32 rows unsplit, 17 to 20 us halved, 20 us in quarters.
template <int kT>
int few_split(int64_t tiles, int64_t blocks)
{
    const int64_t slots = (kT == 64 ? 2 : 1) * static_cast<int64_t>(sm_count());
    int S = 1;
    while (S < 8 && tiles * S * 2 <= slots && 4 * S <= blocks)
        S *= 2;
    return S;
}

// Tiles of kT rows: with one group they are known, otherwise at most so many.
template <int kT>
int64_t few_tiles(const MmArgs &p)
{
    const int64_t nt = (p.N + 127) / 128;
    return (p.offs ? p.M / kT + (p.G < p.M ? p.G : p.M) + 1 : (p.M + kT - 1) / kT) * nt;
}

template <int kT, Mode kMode, Out kOut, Epi kEpi>
fq_status launch_few(const uint8_t *a, const uint8_t *b, int64_t K, const MmArgs &p, cudaStream_t st)
{
    using F = Few<kT, kEpi == kGated>;
    CUtensorMap tx, tw;
    if (!encode_tensor_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, p.M, K, kBlockK, kT,
                              CU_TENSOR_MAP_SWIZZLE_128B, true) ||
        !encode_tensor_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, b, K,
                              static_cast<uint64_t>(p.G) * F::parts * p.N, K, kBlockK, 128,
                              CU_TENSOR_MAP_SWIZZLE_128B, true)) {
        set_last_cuda_error(static_cast<int>(cudaErrorNotSupported));
        return FQ_ERR_CUDA;
    }
    const auto kern = fp8_matmul_few_kernel<kT, kMode, kOut, kEpi>;
    constexpr bool kQuantized = kOut == kE4m3;
    static_assert(few_bytes<kT, kEpi == kGated, kQuantized>(kQuantized ? 371 : 480) <= 113 * 1024,
                  "two CTAs of an SM, as many groups as the comment above says");
    const size_t dyn = few_bytes<kT, kEpi == kGated, kQuantized>(p.G);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(dyn)) != cudaSuccess)
        return launch_status();
    const int64_t tiles = few_tiles<kT>(p), sms = sm_count();
    const int S = few_split<kT>(tiles, p.KB);
    const int64_t most = S > 1 ? tiles : F::per_sm * sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(S * (tiles < most ? tiles : most)));
    cfg.blockDim = dim3(F::threads);
    cfg.dynamicSmemBytes = dyn;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, tx, tw, p, static_cast<int32_t>(S)) != cudaSuccess)
        return launch_status();
    return launch_status();
}

// Whether tiles of one CTA (128 x 128) finish before tiles of a pair (256 x pair_cols):
// rounds over the SMs, a round of one CTA's taking `permille` of a round of pairs.
// Measured both ways: forward 625 (N x K 4096 x 7168, 512 rows: 128 tiles, one round 21.4
// us, pairs 27.0; 1024 rows: 256 tiles, two rounds 37.6, pairs 28.2), weight gradient 520
// (1003 tokens, 8 x 1408 x 2048: 10 rounds 28.1 us, 6 of pairs 30.9; 16384 tokens, 16 x
// 2048 x 2048: 27 rounds 150, 14 of pairs 144).  Gated, where both kinds of tiles have 128
// columns of c and a CTA the same work in them, 1170 (384 x 2 x 14336 x 4096: three rounds
// 58, three of pairs 51; 384 x 2 x 2048 x 20480: one round 82, one of pairs 67; 640 x 2 x
// 13824 x 5120: four 89, five 93; 896 x 2 x 18944 x 3584: seven 112, eight 111).
inline bool one_cta_tiles(int64_t rows, int64_t cols, int64_t groups, int64_t pair_cols,
                          int permille)
{
    const int64_t sms = sm_count(), pairs = sms > 1 ? sms / 2 : 1;
    const int64_t one = (rows + 127) / 128 * ((cols + 127) / 128) * groups;
    const int64_t two = (rows + 255) / 256 * ((cols + pair_cols - 1) / pair_cols) * groups;
    return (one + sms - 1) / sms * permille < (two + pairs - 1) / pairs * 1000;
}

// Which kernel an epilogue runs with where the weights are small (up to 64 MB, so
// that their HBM time hides no difference): rows of a tile of few rows (16, 32, 64), or
// CTAs of a large tile (1, 2), whichever ends first by its time without blocks, that of
// a block, and for few rows what more CTAs than SMs add, and each row whose sums come
// from a cluster's CTAs.  Fitted to the five kernels' times at 14136 random sizes (1 to
// 2500 rows, dense and in up to 64 groups, x 64 to 4096 columns, K 256 to 14336, every form
// of the epilogue): the choice is 0.8 % behind the best of the five on average, 19 % at the
// 99th percentile, and no more at 8742 others.  64 x 2 x 896 x 7168: few rows 9.1 us, one CTA
// a tile 27.7; 100 x 1408 x 1024: 6.0, 8.6; 200 x 4096 x 7168: 22.5, 21.9.
template <Epi kEpi>
int pick_small(const MmArgs &p)
{
    constexpr bool kTwo = kEpi == kGated;
    const int64_t sms = sm_count(), M = p.M, nt = (p.N + 127) / 128;
    const int64_t groups = p.G < M ? p.G : M;
    // row tiles, of ragged groups half of one more for each
    const auto row_tiles = [&](int64_t rows) {
        const int64_t n = p.G == 1 ? (M + rows - 1) / rows : M / rows + groups / 2;
        return n > groups ? n : groups;
    };
    int best = 2;
    int64_t least = INT64_MAX;
    const auto offer = [&](int which, int64_t ns) {
        if (ns < least) {
            least = ns;
            best = which;
        }
    };
    const int64_t mean = (M + p.G - 1) / p.G;
    const auto few = [&](auto rows, int64_t fixed, int64_t block, int64_t many, int64_t row) {
        constexpr int kT = decltype(rows)::value;
        // (split as the launch will split it)
        const int64_t tiles = row_tiles(kT) * nt, S = few_split<kT>(few_tiles<kT>(p), p.KB);
        const int64_t waves = (tiles * S + 2 * sms - 1) / (2 * sms);
        offer(kT, fixed + (tiles * S > sms ? many : 0) +
                      (S > 1 ? (mean < kT ? mean : kT) / S * row : 0) +
                      waves * ((p.KB + S - 1) / S) * block);
    };
    using std::integral_constant;
    few(integral_constant<int, 16>{}, kTwo ? 3450 : 3500, kTwo ? 410 : 270, kTwo ? 1975 : 1025,
        kTwo ? 280 : 310);
    few(integral_constant<int, 32>{}, kTwo ? 4100 : 4600, kTwo ? 415 : 270, kTwo ? 2100 : 1270,
        kTwo ? 290 : 225);
    if (!kTwo)
        few(integral_constant<int, 64>{}, 4800, 495, 875, 270);
    const int64_t wide = kTwo ? nt : (p.N + 255) / 256;
    offer(1, (kTwo ? 6800 : 7350) +
                 (row_tiles(128) * nt + sms - 1) / sms * p.KB * (kTwo ? 390 : 247));
    offer(2, (kTwo ? 8950 : 12050) +
                 (row_tiles(256) * wide + sms / 2 - 1) / (sms / 2) * p.KB * (kTwo ? 370 : 397));
    return best;
}

template <Mode kMode, Out kOut, Epi kEpi>
fq_status launch_forward(const uint8_t *a, const uint8_t *b, int64_t K, const MmArgs &p,
                         cudaStream_t st)
{
    // Which kernel, by the mean rows of a group and the tiles (N x K 4096 x 7168
    // unless said otherwise; us):
    //   rows 32: few rows 9.9, one CTA a tile 19.9, pairs 26.4
    //   rows 64: 12.3 (K split eight ways), 19.9, 26.5; but 14336 x 4096, where it
    //            is not split: 24.0, 14.4, 18.8; 32 groups of 64: 176, 167, 197
    //   32 groups of 128 rows: one CTA a tile 175, pairs 201; of 256: 288, 227
    // The counts themselves are on the device.  4096 rows over 256 groups: 1272 even, 1333
    // with half of them in one group, 1307 with one row in all the others; all in one
    // group 416, where the pairs of a dense product take 102.
    const int64_t mean = (static_cast<int64_t>(p.M) + p.G - 1) / p.G;
    const int64_t sms = sm_count(), nt = (p.N + 127) / 128;
    const int64_t b_rows = static_cast<int64_t>(p.G) * p.N * (kEpi == kGated ? 2 : 1);
    if constexpr (kEpi != kPlain) {
        if (b_rows * K <= 64 << 20) {
            switch (pick_small<kEpi>(p)) {
            case 16:
                return launch_few<16, kMode, kOut, kEpi>(a, b, K, p, st);
            case 32:
                return launch_few<32, kMode, kOut, kEpi>(a, b, K, p, st);
            case 64:
                if constexpr (kEpi != kGated)
                    return launch_few<64, kMode, kOut, kEpi>(a, b, K, p, st);
            case 1:
                return launch_matmul<1, kMode, kOut, kEpi>(a, p.M, b, b_rows, K, p.M, p, st);
            default:
                return launch_matmul<2, kMode, kOut, kEpi>(a, p.M, b, b_rows, K, p.M, p, st);
            }
        }
    }
    // (gated, 16 rows in each of 32 groups on average: tiles of 16 rows 169, of 32 rows,
    // which hold a whole group more often, 164; dense 16 rows x 2 x 14336 x 4096: 27.4, 29.4)
    if (mean <= (kEpi == kGated && p.G > 1 ? 8 : 16))
        return launch_few<16, kMode, kOut, kEpi>(a, b, K, p, st);
    if (mean <= 32)
        return launch_few<32, kMode, kOut, kEpi>(a, b, K, p, st);
    if constexpr (kEpi != kGated)
        if (mean <= 64 && 2 * nt * p.G <= sms)
            return launch_few<64, kMode, kOut, kEpi>(a, b, K, p, st);
    if (p.G > 1 ? mean <= 128
                : one_cta_tiles(p.M, p.N, 1, Shape<2, kOut, kEpi>::step, kEpi == kGated ? 1170 : 625))
        return launch_matmul<1, kMode, kOut, kEpi>(a, p.M, b, b_rows, K, p.M, p, st);
    return launch_matmul<2, kMode, kOut, kEpi>(a, p.M, b, b_rows, K, p.M, p, st);
}

// The checks and arguments that the products share; a status other than FQ_OK
// ends the call, and so does M = 0 (p.M is 0 then).
inline fq_status matmul_args(const uint8_t *a, const float *sa, int64_t M, int64_t K,
                             const uint8_t *b, const float *sb, int64_t N, int b_block,
                             int64_t matrices, const int64_t *group_offsets, int32_t G,
                             const void *c, int32_t *dev_status, MmArgs &p)
{
    if (M < 0 || M > INT32_MAX - 512 || N <= 0 || K <= 0 || K % 128 != 0 || K > INT32_MAX - 128)
        return FQ_ERR_SHAPE;
    if (G < 1 || G > FQ_COLS_MAX_GROUPS || (b_block != 1 && b_block != 128) ||
        (!group_offsets && G != 1))
        return FQ_ERR_ARG;
    // 32-bit rows of b and 32-bit tile indices
    if (N > (INT32_MAX - 512) / (matrices * G) ||
        (M / 128 + G + 2) * (N / 128 + 1) > INT32_MAX / 2)
        return FQ_ERR_SHAPE;
    p = {};
    if (M == 0)
        return FQ_OK;
    if (!a || !sa || !b || !sb || !c)
        return FQ_ERR_NULL;
    if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(c) ||
        !aligned16(group_offsets))
        return FQ_ERR_ALIGN;
    p.sa = sa;
    p.sb = sb;
    p.offs = group_offsets;
    p.c = const_cast<void *>(c);
    p.dev_status = dev_status;
    p.G = G;
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.KB = static_cast<int32_t>(K / 128);
    p.sb_rows = b_block == 1 ? p.N : (p.N + 127) / 128;
    return FQ_OK;
}

}  // namespace

}  // namespace fq
