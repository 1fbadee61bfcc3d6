// Launchers and shared types of the attention kernels
// (include/spgemm_attention.h).
#pragma once

#include "../../include/spgemm_attention.h"
#include "attention_tile.h"
#include "common.h"

namespace sg {

// A piece of one row of the mask (or of its transpose): the work of one
// wavefront per key head. slot is where its partial result goes, -1 if it is
// the whole row and so writes the result itself.
struct AttnPiece {
    int64_t first;  // first entry
    int32_t row;
    int32_t len;    // entries; 0 only for a row without any
    int32_t slot;
    int32_t lead;   // 1 for the first piece of its row
};
// A row of more than one piece: the slots that make it up.
struct AttnSplit {
    int32_t row;
    int32_t slot;
    int32_t count;
    int32_t pad;
};

// One direction of the mask, cut into pieces.
struct AttnSide {
    int64_t n = 0;          // rows, or blocks of rows
    int64_t npieces = 0;
    int64_t nslots = 0;
    int64_t nsplits = 0;
    const AttnPiece* pieces = nullptr;
    const AttnSplit* splits = nullptr;
    const int32_t* idx = nullptr;  // the entries' columns
    const uint16_t* bits = nullptr;  // see kColBlock and kRowBlock; null for single rows
    int block = 1;                   // rows per block
};

// The transposed mask, by blocks of 16 columns: an entry of block b is a row
// (idx) with the set of the block's columns that the row stores (bits), so
// that one trip for the row's q and dout serves up to 16 keys. Within a block
// rows ascend; a row comes again where it stores a column twice, or columns
// out of order.
constexpr int kColBlock = 16;
// The mask by blocks of 4 rows, in the same manner: an entry is a column with
// the set of the block's rows that store it, so that one trip for its key and
// value rows serves up to 4 rows, and 4 short rows share a tile.
constexpr int kRowBlock = 4;

// Rows of a gathered tensor. A row's offset is unit * (its index) << shift
// bytes, so that it fits 32 bits before the shift; the strides of every
// dimension are multiples of 1 << shift.
struct AttnGather {
    const char* base = nullptr;
    int64_t head = 0;   // bytes between heads
    uint32_t unit = 0;
    uint32_t shift = 0;
};
struct AttnRows {
    char* base = nullptr;
    int64_t row = 0;    // bytes between rows
    int64_t head = 0;
};

struct AttnShape {
    int type = 0;
    int hq = 0, hkv = 0, group = 0, dim = 0;
    int mtiles = 1;      // tiles of 16 queries per piece and key head (see AttnColumn)
    float scale = 0.f;   // of the scores
    float c = 0.f;       // scale * log2(e)
    float c_low = 0.f;   // and what c rounds off
    float mag = 1.f;     // |c|, or 1 if that is 0: the factor that Softmax takes
};

struct ForwardArgs {
    AttnShape s;
    AttnSide side;
    int64_t nrows = 0;
    AttnRows q, out;
    AttnGather k, v;
    float* lse = nullptr;      // may be null
    float* part = nullptr;     // [slot][row of block][hq][dim] unnormalised outputs
    float* part_ml = nullptr;  // [slot][row of block][hq][2]: maximum (base 2) and sum
};
void attention_forward(const ForwardArgs& a, hipStream_t st);

struct BackwardArgs {
    AttnShape s;
    AttnSide rows, cols;
    AttnRows q, out, dout, dq, dk, dv;
    AttnGather k, v;        // gathered by the row pass
    AttnGather gq, gdout;   // q and dout, gathered by the column pass
    AttnRows krow, vrow;    // k and v, one row per column of the mask
    const float* lse = nullptr;
    float* delta = nullptr;    // [row][hq]
    float* part_q = nullptr;   // [slot][row of block][hq][dim]
    float* part_kv = nullptr;  // [slot of cols][hkv][kColBlock][2][dim]
    int64_t nrows = 0, ncols = 0;
    FastDiv group_div;
};
void attention_backward(const BackwardArgs& a, hipStream_t st);

struct PagedArgs {
    AttnShape s;
    AttnRows q, out;
    const char* k = nullptr;
    const char* v = nullptr;
    // offsets in units of 1 << shift bytes, as AttnGather
    uint32_t k_page = 0, k_slot = 0, v_page = 0, v_slot = 0;
    uint32_t k_shift = 0, v_shift = 0;
    int64_t k_head = 0, v_head = 0;  // bytes
    int64_t npages = 0;
    FastDiv page_div, group_div;
    int64_t seqs = 0, tokens = 0, room = 0;  // room: entries of col
    const int64_t* rowptr = nullptr;
    const int32_t* col = nullptr;
    const int64_t* q_rowptr = nullptr;
    const int64_t* lengths = nullptr;
    int32_t max_new = 0, max_length = 0;
    // Keys per piece, a multiple of 32, and ceil(max_length / piece); where keys are not
    // cut, or cut in ranges, one piece that holds all (max_length, whatever it divides).
    int32_t piece = 0;
    int32_t npieces = 1;
    int32_t ranges = 0;    // not 0: EvenSplit's, instead of pieces
    float* lse = nullptr;
    // Rows' parts, as pieces [piece][token][hq], as ranges [2 range + late][key head]
    // [tile][row of the tile]: of each dim values, and its maximum and sum.
    float* part = nullptr;
    float* part_ml = nullptr;
};
void paged_attention(const PagedArgs& a, hipStream_t st);
// Joins the pieces of every token and query head (npieces > 1).
void paged_join(const PagedArgs& a, hipStream_t st);
// Whether a work group shares the keys of a sequence's `rows` rows (new
// tokens times the query heads of a key head), and the rows of its tiles.
bool paged_wide(const AttnShape& s, int64_t rows);
constexpr int kPagedTileMost = 128;
int paged_tile_rows(const AttnShape& s, int64_t rows);

// The grid of at least that many work groups, which kernels number along x, then
// y. A launch whose lanes along one axis pass 2^32 runs without those past it and
// without an error.
inline dim3 grid_2d(int64_t blocks) {
    constexpr int64_t most = int64_t(1) << 22;  // of up to 512 lanes
    if (blocks <= most) return dim3(grid_1d(blocks));
    const int64_t y = ceil_div(blocks, most);
    if (y > 65535) throw OverflowError("grid size exceeds the HIP limit");
    return dim3((unsigned)most, (unsigned)y);
}
__device__ __forceinline__ int64_t grid_block() {
    return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

// XCD x of the 8 gets every eighth work group; this gives each XCD a
// contiguous eighth of the logical blocks, so that neighbouring pieces of one
// head, which gather the same key rows, meet in one XCD's L2.
constexpr int kXcds = 8;
inline int64_t xcd_grid(int64_t blocks) { return ceil_div(blocks, kXcds) * kXcds; }
__device__ __forceinline__ int64_t xcd_block() {
    const int64_t per = (int64_t)gridDim.x / kXcds * gridDim.y;
    return (int64_t)(blockIdx.x % kXcds) * per + grid_block() / kXcds;
}

// Pieces that one wavefront takes in turn: enough to hide the first trip to
// memory of each but the first, few enough that the chip's about 3000
// wavefronts are replaced several times over (the pieces differ in length).
inline int pieces_per_wave(int64_t units) {
    const int64_t n = units / 12288;
    return (int)(n < 1 ? 1 : n > 16 ? 16 : n);
}

// A wavefront's pieces, the i-th one's record in lane i, and the stream of
// their tiles: the cursor names a tile and moves on to the next piece's first
// one. Empty pieces are not in the stream.
struct PieceStream {
    struct Cursor {
        int i, t0, len;
        uint64_t first;
        bool more;
    };
    AttnPiece mine{};
    uint64_t empty, todo;
    const int32_t* idx;
    const uint16_t* bits;

    __device__ __forceinline__ PieceStream(const AttnSide& side, int64_t first, int stride,
                                           int each)
        : idx(side.idx), bits(side.bits) {
        const int64_t u = first + (int64_t)lane_id() * stride;
        const bool there = lane_id() < each && u < side.npieces;
        if (there) mine = side.pieces[u];
        empty = __ballot(there && mine.len == 0);
        todo = __ballot(there && mine.len > 0);
    }
    static __device__ __forceinline__ int lane_value(int v, int i) {
        return __builtin_amdgcn_readlane(v, i);
    }
    __device__ __forceinline__ int row(int i) const { return lane_value(mine.row, i); }
    __device__ __forceinline__ int slot(int i) const { return lane_value(mine.slot, i); }
    __device__ __forceinline__ int lead(int i) const { return lane_value(mine.lead, i); }
    __device__ __forceinline__ void open(Cursor& c) {
        c.more = todo != 0;
        if (!c.more) return;
        c.i = __builtin_ctzll(todo);
        todo &= todo - 1;
        c.t0 = 0;
        c.len = lane_value(mine.len, c.i);
        const uint32_t lo = (uint32_t)lane_value((int)(mine.first & 0xffffffff), c.i);
        const uint32_t hi = (uint32_t)lane_value((int)(mine.first >> 32), c.i);
        c.first = (uint64_t)hi << 32 | lo;
    }
    __device__ __forceinline__ void next(Cursor& c, int tile) {
        c.t0 += tile;
        if (c.t0 >= c.len) open(c);
    }
    // This lane's entry of the tile. Lanes past the piece's end repeat its
    // last one: every address made from an index is a row that the piece
    // names. Their bits are 0.
    struct Entry {
        uint32_t id, bits;
    };
    template <bool SHARED>
    __device__ __forceinline__ Entry entry(const Cursor& c, int tile) const {
        const int at = c.t0 + (lane_id() & (tile - 1));
        const uint64_t e = c.first + min(at, c.len - 1);
        Entry x{(uint32_t)idx[e], 0};
        if constexpr (SHARED) x.bits = at < c.len ? bits[e] : 0;
        return x;
    }
};

// Which query this lane (and the three that share l % 16) has in tile mt of a
// piece: 16 query heads of one row, or with blocks of rows the query heads of
// block / mtiles rows of the block.
struct AttnColumn {
    bool has;
    int rr, hq;  // row of the block, query head
    __device__ __forceinline__ AttnColumn(const AttnShape& s, int block, int h, int mt) {
        const int n = lane_id() & 15;
        if (block == 1) {
            rr = 0;
            hq = h * s.group + 16 * mt + n;
            has = 16 * mt + n < s.group;
        } else {
            const int rows = block / s.mtiles, r = n / s.group;
            rr = mt * rows + r;
            hq = h * s.group + n - r * s.group;
            has = r < rows;
        }
    }
    // The keys of a tile that the column's row stores, from each lane's bits.
    __device__ __forceinline__ Seen seen(uint32_t bits) const {
        uint32_t all = 0;
#pragma unroll
        for (int r = 0; r < kRowBlock; ++r) {
            const uint32_t b = (uint32_t)__ballot(bits >> r & 1);
            all = rr == r ? b : all;
        }
        return Seen::keys(all);
    }
};

template <class F>
void with_type(int type, int dim, F&& f) {
    if (type == SPGEMM_TYPE_BF16) with_dim<__bf16>(dim, f);
    else if (type == SPGEMM_TYPE_F16) with_dim<_Float16>(dim, f);
    else with_dim<float>(dim, f);
}

}  // namespace sg
