// Plans of attention over a CSR mask, argument checks, and the C ABI of
// include/spgemm_attention.h.
#include <memory>

#include "attention_checks.h"
#include "kernels.h"
#include "primitives.h"

using namespace sg;

struct spgemm_attention_plan_s {
    int device = 0;
    int64_t nrows = 0, ncols = 0, nnz = 0;
    bool backward = false;
    AttnSide rows;    // single rows
    AttnSide blocks;  // blocks of rows, if built (n > 0)
    bool overlap = false;  // the blocks' entries are at most half of the rows'
    AttnSide cols;    // blocks of 16 columns
    AttnSide cut_cols;  // the same in shorter pieces, for few key heads
    void* slab = nullptr;  // what ar's buffers lie in, if not in allocations of their own
    Arena ar;              // pieces, splits and entries; never changed after creation
    ~spgemm_attention_plan_s() {
        ar.release();
        if (slab) (void)hipFree(slab);
    }
};

namespace {

// ---------------------------------------------------------------- plan
// Entries per piece. Rows are cut where they are longer than twice the mean, so
// that rows of about one length stay whole (a cut one's pieces are written and
// joined in floats), or longer than all entries spread over the chip: then
// the longest would end last. (`share` entries of every piece's worth: with
// some 4 key heads, 512 wavefronts' or 192 work groups' share each.)
struct PieceRule {
    int64_t share, least;
    int64_t length(int64_t n, int64_t entries) const {
        const int64_t twice = ceil_div(2 * entries, n < 1 ? 1 : n);
        int64_t want = std::min(twice, ceil_div(entries, share));
        want = ceil_div(want, 32) * 32;
        return want < least ? least : want > 1024 ? 1024 : want;
    }
};
constexpr PieceRule kRowPieces{512, 64}, kBlockPieces{192, 32}, kShortPieces{1024, 32};

struct RowPieces {
    const int64_t* rp;
    int64_t len;
    __host__ __device__ int64_t count(int64_t i) const {
        const int64_t n = rp[i + 1] - rp[i];
        return n <= len ? 1 : (n + len - 1) / len;
    }
    __device__ int64_t operator()(int64_t i) const { return count(i); }
};
struct RowSlots {
    RowPieces p;
    __device__ int64_t operator()(int64_t i) const {
        const int64_t c = p.count(i);
        return c > 1 ? c : 0;
    }
};
struct RowSplit {
    RowPieces p;
    __device__ int64_t operator()(int64_t i) const { return p.count(i) > 1 ? 1 : 0; }
};

__global__ void k_fill_pieces(RowPieces rows, int64_t n, const int64_t* piece0,
                              const int64_t* slot0, const int64_t* split0, AttnPiece* pieces,
                              AttnSplit* splits, int64_t npieces) {
    const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (g >= npieces) return;
    const int64_t row = upper_index(piece0, int64_t(0), n, g);
    const int64_t b = rows.rp[row], e = rows.rp[row + 1];
    const int64_t count = piece0[row + 1] - piece0[row], k = g - piece0[row];
    // equal pieces, of whole tiles
    const int64_t each = ((e - b + count - 1) / count + 31) / 32 * 32;
    AttnPiece p;
    p.first = min(b + k * each, e);
    p.row = (int32_t)row;
    p.len = (int32_t)min(each, e - p.first);
    p.slot = count > 1 ? (int32_t)(slot0[row] + k) : -1;
    p.lead = k == 0;
    pieces[g] = p;
    if (count > 1 && k == 0) splits[split0[row]] = {(int32_t)row, p.slot, (int32_t)count, 0};
}

__global__ void k_entry_rows(const int64_t* rp, int64_t n, int64_t nnz, int32_t* row) {
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e < nnz) row[e] = (int32_t)upper_index(rp, int64_t(0), n, e);
}
__global__ void k_iota(int32_t* x, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) x[i] = (int32_t)i;
}
__global__ void k_gather(const int32_t* src, const int32_t* perm, int64_t n, int32_t* dst) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) dst[i] = src[perm[i]];
}
struct BlockDigit {
    const int32_t* col;
    const int32_t* entry;
    int shift;
    __device__ int operator()(int64_t i) const { return (col[entry[i]] >> shift) & 15; }
};

// Entries in the order (column block, row, place in the row). An entry
// begins a new group where the block or the row changes, or the column does
// not ascend: a group's columns differ, so 16 bits hold them.
struct GroupStart {
    const int32_t* col;
    const int32_t* row;
    const int32_t* entry;
    __device__ int64_t operator()(int64_t i) const {
        if (i == 0) return 1;
        const int32_t e = entry[i], f = entry[i - 1];
        return col[e] / kColBlock != col[f] / kColBlock || row[e] != row[f] || col[e] <= col[f];
    }
};
__global__ void k_fill_groups(GroupStart g, int64_t nnz, const int64_t* group, int32_t* idx,
                              uint16_t* bits) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= nnz || g(i) == 0) return;
    uint32_t m = 0;
    for (int64_t j = i; j < nnz && (j == i || g(j) == 0); ++j)
        m |= 1u << (g.col[g.entry[j]] % kColBlock);
    idx[group[i]] = g.row[g.entry[i]];
    bits[group[i]] = (uint16_t)m;
}
// First group of every block, and the groups' number behind the last.
__global__ void k_block_groups(const int32_t* col, const int32_t* entry, int64_t nnz,
                               const int64_t* group, int64_t nblocks, int64_t* first) {
    const int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (b > nblocks) return;
    int64_t lo = 0, hi = nnz;  // first entry of block b or later
    while (lo < hi) {
        const int64_t mid = lo + ((hi - lo) >> 1);
        if (col[entry[mid]] / kColBlock < b) lo = mid + 1; else hi = mid;
    }
    first[b] = group[lo];
}

// First entry from lo on, before hi, of a row with ascending columns that is
// not below c.
__device__ __forceinline__ int64_t lower_index(const int32_t* col, int64_t lo, int64_t hi,
                                               int32_t c) {
    while (lo < hi) {
        const int64_t mid = lo + ((hi - lo) >> 1);
        if (col[mid] < c) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// lead[e] = 1 if no earlier row of entry e's block stores its column; *flag is
// set where a row's columns do not ascend.
__global__ void k_block_leaders(const int64_t* rp, const int32_t* col, const int32_t* row,
                                int64_t nnz, int32_t* lead, int* flag) {
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= nnz) return;
    const int32_t r = row[e], c = col[e];
    if (e > rp[r] && col[e - 1] >= c) *flag = 1;  // (every writer writes the same)
    int32_t is = 1;
    for (int32_t x = r / kRowBlock * kRowBlock; x < r && is; ++x) {
        const int64_t end = rp[x + 1], at = lower_index(col, rp[x], end, c);
        if (at < end && col[at] == c) is = 0;
    }
    lead[e] = is;
}
// The blocks' entries in the order of their columns. before[e]: leaders among
// the entries below e; a leader's place is its block's first plus the number
// of the block's leaders with smaller columns.
__global__ void k_block_entries(const int64_t* rp, int64_t n, const int32_t* col,
                                const int32_t* row, int64_t nnz, const int32_t* lead,
                                const int64_t* before, int32_t* idx, uint16_t* bits) {
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= nnz || !lead[e]) return;
    const int32_t c = col[e];
    const int64_t r0 = row[e] / kRowBlock * kRowBlock;
    int64_t place = before[rp[r0]];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRowBlock; ++i) {
        if (r0 + i >= n) break;
        const int64_t b = rp[r0 + i], end = rp[r0 + i + 1], at = lower_index(col, b, end, c);
        place += before[at] - before[b];
        if (at < end && col[at] == c) m |= 1u << i;
    }
    idx[place] = c;
    bits[place] = (uint16_t)m;
}
__global__ void k_block_starts(const int64_t* rp, int64_t n, const int64_t* before, int64_t nblocks,
                               int64_t* first) {
    const int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (b <= nblocks) first[b] = before[rp[b * kRowBlock < n ? b * kRowBlock : n]];
}
struct LoadI32 {
    const int32_t* p;
    __device__ int64_t operator()(int64_t i) const { return p[i]; }
};

AttnSide make_side(const char* name, const int64_t* rp, int64_t n, int64_t nnz, PieceRule rule,
                   const int32_t* idx, Arena& keep, Arena& tmp, hipStream_t st) {
    AttnSide s;
    s.n = n;
    s.idx = idx;
    if (n == 0) return s;
    const std::string nm(name);
    const RowPieces rows{rp, rule.length(n, nnz)};
    int64_t* piece0 = tmp.get<int64_t>("piece0", (size_t)n + 1);
    int64_t* slot0 = tmp.get<int64_t>("slot0", (size_t)n + 1);
    int64_t* split0 = tmp.get<int64_t>("split0", (size_t)n + 1);
    scan_exclusive(rows, n, piece0, tmp, st);
    scan_exclusive(RowSlots{rows}, n, slot0, tmp, st);
    scan_exclusive(RowSplit{rows}, n, split0, tmp, st);
    int64_t tot[3];
    SG_HIP(hipMemcpyAsync(&tot[0], piece0 + n, 8, hipMemcpyDeviceToHost, st));
    SG_HIP(hipMemcpyAsync(&tot[1], slot0 + n, 8, hipMemcpyDeviceToHost, st));
    SG_HIP(hipMemcpyAsync(&tot[2], split0 + n, 8, hipMemcpyDeviceToHost, st));
    SG_HIP(hipStreamSynchronize(st));
    s.npieces = tot[0];
    s.nslots = tot[1];
    s.nsplits = tot[2];
    if (s.npieces > 0x7fffffffLL) throw OverflowError("more pieces than supported");
    AttnPiece* pieces = static_cast<AttnPiece*>(
        keep.get(nm + "_pieces", (size_t)s.npieces * sizeof(AttnPiece)));
    AttnSplit* splits = static_cast<AttnSplit*>(
        keep.get(nm + "_splits", (size_t)s.nsplits * sizeof(AttnSplit)));
    hipLaunchKernelGGL(k_fill_pieces, dim3(grid_1d(ceil_div(s.npieces, 256))), dim3(256), 0, st,
                       rows, n, piece0, slot0, split0, pieces, splits, s.npieces);
    SG_LAUNCH_CHECK();
    s.pieces = pieces;
    s.splits = splits;
    return s;
}

// Blocks of 4 rows, where they serve: the rows are short (they share tiles) or
// store the same columns (they share keys), and their columns ascend (else
// the blocks stay unbuilt and single rows do). 4 heads to a key head, 8192 rows of
// 128 spread keys: 159 us by blocks and 172 by rows; of 256 keys 277 by either.
bool blocks_serve(int64_t n, int64_t nnz, int64_t entries) {
    return nnz < 192 * n || entries <= nnz / 4 * 3;
}
void build_blocks(spgemm_attention_plan p, const DevCSR& m, const int32_t* col, const int32_t* row,
                  Arena& tmp, hipStream_t st) {
    const unsigned g = grid_1d(ceil_div(m.nnz, 256));
    const int64_t nblocks = ceil_div(m.n, kRowBlock);
    int32_t* lead = tmp.get<int32_t>("lead", (size_t)m.nnz);
    int64_t* before = tmp.get<int64_t>("before", (size_t)m.nnz + 1);
    int* flag = tmp.get<int>("flag", 1);
    fill<int>(flag, 1, 0, st);
    hipLaunchKernelGGL(k_block_leaders, dim3(g), dim3(256), 0, st, m.rp, col, row, m.nnz, lead,
                       flag);
    SG_LAUNCH_CHECK();
    scan_exclusive(LoadI32{lead}, m.nnz, before, tmp, st);
    int unsorted = 0;
    int64_t entries = 0;
    SG_HIP(hipMemcpyAsync(&unsorted, flag, sizeof(int), hipMemcpyDeviceToHost, st));
    SG_HIP(hipMemcpyAsync(&entries, before + m.nnz, 8, hipMemcpyDeviceToHost, st));
    SG_HIP(hipStreamSynchronize(st));
    if (unsorted || !blocks_serve(m.n, m.nnz, entries)) return;
    int32_t* idx = p->ar.get<int32_t>("block_idx", (size_t)entries);
    uint16_t* bits = p->ar.get<uint16_t>("block_bits", (size_t)entries);
    int64_t* first = tmp.get<int64_t>("block_first", (size_t)nblocks + 1);
    hipLaunchKernelGGL(k_block_entries, dim3(g), dim3(256), 0, st, m.rp, m.n, col, row, m.nnz, lead,
                       before, idx, bits);
    SG_LAUNCH_CHECK();
    hipLaunchKernelGGL(k_block_starts, dim3(grid_1d(ceil_div(nblocks + 1, 256))), dim3(256), 0, st,
                       m.rp, m.n, before, nblocks, first);
    SG_LAUNCH_CHECK();
    p->blocks = make_side("blocks", first, nblocks, entries, kRowPieces, idx, p->ar, tmp, st);
    p->blocks.bits = bits;
    p->blocks.block = kRowBlock;
    p->overlap = entries <= m.nnz / 2;
}

// The transposed mask by blocks of columns.
void build_cols(spgemm_attention_plan p, const DevCSR& m, const int32_t* col, const int32_t* row,
                Arena& tmp, hipStream_t st) {
    const int64_t nblocks = ceil_div(m.m, kColBlock);
    int64_t* first = tmp.get<int64_t>("first", (size_t)nblocks + 1);
    int32_t* gidx = p->ar.get<int32_t>("groups", (size_t)m.nnz);
    uint16_t* gbits = p->ar.get<uint16_t>("bits", (size_t)m.nnz);
    int64_t ngroups = 0;
    if (m.nnz > 0) {
        // a stable radix sort of the entries by column block, 4 bits a pass:
        // rows ascend within a block, so its sums have one order
        const unsigned g = grid_1d(ceil_div(m.nnz, 256));
        int32_t* cur = tmp.get<int32_t>("cur", (size_t)m.nnz);
        int32_t* next = tmp.get<int32_t>("next", (size_t)m.nnz);
        int32_t* perm = tmp.get<int32_t>("perm", (size_t)m.nnz);
        int64_t* bins = tmp.get<int64_t>("bins", 17);
        int64_t* group = tmp.get<int64_t>("group", (size_t)m.nnz + 1);
        hipLaunchKernelGGL(k_iota, dim3(g), dim3(256), 0, st, cur, m.nnz);
        SG_LAUNCH_CHECK();
        for (int shift = ilog2(kColBlock); shift < 31 && (m.m - 1) >> shift > 0; shift += 4) {
            partition(BlockDigit{col, cur, shift}, m.nnz, 16, perm, nullptr, bins, tmp, st);
            hipLaunchKernelGGL(k_gather, dim3(g), dim3(256), 0, st, cur, perm, m.nnz, next);
            SG_LAUNCH_CHECK();
            std::swap(cur, next);
        }
        const GroupStart start{col, row, cur};
        scan_exclusive(start, m.nnz, group, tmp, st);
        hipLaunchKernelGGL(k_fill_groups, dim3(g), dim3(256), 0, st, start, m.nnz, group, gidx,
                           gbits);
        SG_LAUNCH_CHECK();
        hipLaunchKernelGGL(k_block_groups, dim3(grid_1d(ceil_div(nblocks + 1, 256))), dim3(256), 0,
                           st, col, cur, m.nnz, group, nblocks, first);
        SG_LAUNCH_CHECK();
        SG_HIP(hipMemcpyAsync(&ngroups, group + m.nnz, 8, hipMemcpyDeviceToHost, st));
        SG_HIP(hipStreamSynchronize(st));
    } else {
        fill<int64_t>(first, nblocks + 1, 0, st);
    }
    p->cols = make_side("cols", first, nblocks, ngroups, kBlockPieces, gidx, p->ar, tmp, st);
    p->cols.bits = gbits;
    p->cols.block = kColBlock;
    p->cut_cols = p->cols;
    if (kShortPieces.length(nblocks, ngroups) < kBlockPieces.length(nblocks, ngroups)) {
        p->cut_cols = make_side("cut_cols", first, nblocks, ngroups, kShortPieces, gidx, p->ar,
                                tmp, st);
        p->cut_cols.bits = gbits;
        p->cut_cols.block = kColBlock;
    }
}

// Device memory given back with the scope.
struct Slab {
    void* p = nullptr;
    explicit Slab(size_t bytes) {
        if (hipMalloc(&p, bytes) != hipSuccess) {
            (void)hipGetLastError();
            throw OomError("attention plan");
        }
    }
    ~Slab() {
        if (p) (void)hipFree(p);
    }
};

// Bytes that cover a plan's buffers, and those used while it is made: each is
// carved out of one allocation, because allocating and freeing two dozen
// buffers takes longer than the kernels do. A mask so large that the bounds
// are far from the need gets allocations one by one instead.
constexpr int64_t kSlabMost = int64_t(1) << 30;
int64_t kept_bytes(int64_t n, int64_t m, int64_t nnz, bool backward) {
    const int64_t row_cuts = nnz / kRowPieces.least + 1, col_cuts = nnz / kBlockPieces.least + 1;
    int64_t b = 10 * nnz + sizeof(AttnPiece) * (n + n / kRowBlock + 1 + 2 * row_cuts) +
                2 * sizeof(AttnSplit) * row_cuts;
    if (backward)
        b += 6 * nnz + 2 * sizeof(AttnPiece) * (m / kColBlock + 1 + col_cuts) +
             2 * sizeof(AttnSplit) * col_cuts;
    return b + (int64_t(16) << 10);
}
int64_t temporary_bytes(int64_t n, int64_t m, int64_t nnz, bool backward) {
    return (backward ? 37 : 17) * nnz + 40 * n + (backward ? 3 * m : 0) + (int64_t(256) << 10);
}

int build_plan(spgemm_attention_plan p, const spgemm_csr* mask, bool backward, bool slabs,
               hipStream_t st) {
    const int64_t n = mask->nrows, cols = mask->ncols, nnz = mask->nnz;
    const int64_t kept = kept_bytes(n, cols, nnz, backward);
    const int64_t used = temporary_bytes(n, cols, nnz, backward);
    Arena tmp;
    std::unique_ptr<Slab> slab;
    if (slabs && used <= kSlabMost) {
        slab = std::make_unique<Slab>((size_t)used);
        tmp.use_region(slab->p, (size_t)used);
        if (hipMalloc(&p->slab, (size_t)kept) != hipSuccess) {
            (void)hipGetLastError();
            p->slab = nullptr;
            throw OomError("attention plan");
        }
        p->ar.use_region(p->slab, (size_t)kept);
    }
    DevCSR m;
    m.n = mask->nrows;
    m.m = mask->ncols;
    m.nnz = mask->nnz;
    m.rp = mask->rowptr;
    m.col = mask->col;
    int* flag = tmp.get<int>("flag", 1);
    fill<int>(flag, 1, 0, st);
    launch_validate(m, flag, st);
    int bad = 0;
    SG_HIP(hipMemcpyAsync(&bad, flag, sizeof(int), hipMemcpyDeviceToHost, st));
    SG_HIP(hipStreamSynchronize(st));
    if (bad) return SPGEMM_ERR_INDEX_RANGE;
    p->nrows = m.n;
    p->ncols = m.m;
    p->nnz = m.nnz;
    p->backward = backward;
    int32_t* col = p->ar.get<int32_t>("col", (size_t)m.nnz);
    copy<int32_t>(col, m.col, m.nnz, st);
    int32_t* row = tmp.get<int32_t>("row", (size_t)m.nnz);
    if (m.nnz > 0) {
        hipLaunchKernelGGL(k_entry_rows, dim3(grid_1d(ceil_div(m.nnz, 256))), dim3(256), 0, st,
                           m.rp, m.n, m.nnz, row);
        SG_LAUNCH_CHECK();
    }
    p->rows = make_side("rows", m.rp, m.n, m.nnz, kRowPieces, col, p->ar, tmp, st);
    if (m.nnz > 0) build_blocks(p, m, col, row, tmp, st);
    if (backward) build_cols(p, m, col, row, tmp, st);
    SG_HIP(hipStreamSynchronize(st));  // before the temporary buffers go
    return SPGEMM_OK;
}

// The rows' side for a call, and its tiles of 16 queries: blocks of 4 rows
// where their queries fill one tile, or two that mostly see the same keys.
// bf16, 128 values a head, by blocks and by single rows: 4 query heads to a key
// head, 509 K entries of 16384 rows by a power law 270 and 318 us, a window of
// 256 48 and 132 us, 8192 rows of 24 spread keys 53 and 61 us; 8 heads, a window
// of 256 88 and 136 us, but 8192 rows of 64 spread keys 184 and 119 us.
const AttnSide& row_side(spgemm_attention_plan p, AttnShape* s) {
    const bool blocks = p->blocks.n > 0 && (s->group <= 4 || (s->group <= 8 && p->overlap));
    s->mtiles = blocks ? (s->group <= 4 ? 1 : 2) : (s->group + 15) / 16;
    return blocks ? p->blocks : p->rows;
}

// The columns' side for a call: in shorter pieces where the others' work groups,
// one for each of the key heads, are not the three or four per compute unit that
// the chip holds at once (a mask of 1500 x 4000 with 200 entries to a row, heads
// of 128: with 16 query heads on 2 key heads 394 -> 284 us; with 8 on 8, and
// work groups enough, short pieces take 279 us for 263, as their sums go
// through memory).
const AttnSide& col_side(spgemm_attention_plan p, int hkv) {
    return p->cols.npieces * hkv <= 1024 ? p->cut_cols : p->cols;
}

// ---------------------------------------------------------------- checks
// heads = 1: the head is added to the base by the kernel, in 64 bits.
bool make_gather(const AttnRows& r, int64_t n, int64_t heads, AttnGather* g) {
    const int64_t strides[2] = {r.row, r.head}, counts[2] = {n, heads};
    g->base = r.base;
    g->head = r.head;
    if (!gather_unit(strides, counts, 2, &g->shift)) return false;
    g->unit = (uint32_t)(r.row >> g->shift);
    return true;
}

int64_t carve_forward(spgemm_attention_plan p, AttnShape s, void* ws, ForwardArgs* a) {
    const AttnSide& side = row_side(p, &s);
    Carver c{static_cast<char*>(ws)};
    a->part = c.take((__int128)side.nslots * side.block * s.hq * s.dim);
    a->part_ml = c.take((__int128)side.nslots * side.block * s.hq * 2);
    return c.used;
}
int64_t carve_backward(spgemm_attention_plan p, AttnShape s, void* ws, BackwardArgs* a) {
    const AttnSide& side = row_side(p, &s);
    Carver c{static_cast<char*>(ws)};
    a->delta = c.take((__int128)p->nrows * s.hq);
    a->part_q = c.take((__int128)side.nslots * side.block * s.hq * s.dim);
    a->part_kv = c.take((__int128)col_side(p, s.hkv).nslots * s.hkv * kColBlock * 2 * s.dim);
    return c.used;
}

bool plan_here(spgemm_attention_plan p) {
    int dev = -1;
    return hipGetDevice(&dev) == hipSuccess && dev == p->device;
}

// ---------------------------------------------------------------- paged
// Keys per piece. Where there are few rows the keys are cut until there are as
// many wavefronts with keys of their own, or work groups that share keys, as the
// chip holds at once: of the first eight to a compute unit (four from 129 values
// per head on), with at least 64 keys each, of the second two (one), with at
// least 256 keys each, as their pieces cost more to join. (Twice as many of the
// first are no better loaded and have twice the pieces to join: the next token
// of 64 sequences of 8.5 K tokens, 64 heads on 8, 503 us for 468; of 16
// sequences, 16 heads of 256 on 2, 93 us for 52 with four times as many. Half as
// many take 534 us of the former.)
// Twice as many where the batch's chunks differ and are of several tiles, for
// then its texts differ too, and the longest would end last (16 chunks of up
// to 128 tokens, 7 heads of 64: 88 -> 59 us; 8 chunks of up to 8 tokens, one
// tile each, take 55 us, and 64 us if cut so).
void shape_pieces(PagedArgs* a) {
    const int64_t rows = (int64_t)a->max_new * a->s.group;
    const bool wide = paged_wide(a->s, rows);
    const int64_t tile = paged_tile_rows(a->s, rows);
    const int64_t whole_tiles = a->seqs * ceil_div(rows, tile);
    const int64_t tiles = std::min(whole_tiles, a->seqs + a->tokens * a->s.group / tile);
    const bool ragged = rows > tile && a->tokens * 4 < a->seqs * a->max_new * 3;
    const int64_t units = std::max<int64_t>(a->s.hkv * tiles, 1);
    const int64_t most = std::max<int64_t>(ceil_div(a->max_length, wide ? 256 : 64), 1);
    const int64_t target = (a->s.dim <= 128 ? 2 : 1) * (!wide ? 1024 : ragged ? 512 : 256);
    const int64_t want = std::min(std::max<int64_t>(target / units, 1), most);
    const int64_t step = wide ? 64 : 32;
    a->piece = (int32_t)std::max<int64_t>(
        ceil_div(ceil_div(a->max_length, want), step) * step, step);
    a->npieces = (int32_t)std::max<int64_t>(ceil_div(a->max_length, a->piece), 1);
}

int64_t carve_paged(void* ws, PagedArgs* a) {
    Carver c{static_cast<char*>(ws)};
    if (a->npieces > 1) {
        const __int128 rows = (__int128)a->npieces * a->tokens * a->s.hq;
        a->part = c.take(rows * a->s.dim);
        a->part_ml = c.take(rows * 2);
    }
    return c.used;
}

void batch_sizes(const spgemm_paged_batch* b, PagedArgs* a) {
    a->seqs = b->pages->nrows;
    a->tokens = b->tokens;
    a->max_new = (int32_t)std::min(b->max_new, b->tokens);
    a->max_length = (int32_t)b->max_length;
    shape_pieces(a);
}


}  // namespace

extern "C" {

SPGEMM_API int spgemm_attention_plan_create(spgemm_attention_plan* out, const spgemm_csr* mask,
                                            int32_t backward, void* stream) {
    if (!out) return SPGEMM_ERR_INVALID_ARG;
    *out = nullptr;
    if (!mask || mask->nrows < 0 || mask->ncols < 0 || mask->nnz < 0 || !mask->rowptr ||
        (mask->nnz > 0 && !mask->col))
        return SPGEMM_ERR_INVALID_ARG;
    if (mask->ncols > 0x7fffffffLL || mask->nrows >= 0x7fffffffLL || mask->nnz > 0x7fffffffLL)
        return SPGEMM_ERR_OVERFLOW;
    spgemm_attention_plan p = nullptr;
    const int rc = guarded([&]() -> int {
        int device = 0;
        SG_HIP(hipGetDevice(&device));
        for (const bool slabs : {true, false}) {
            delete p;
            p = nullptr;
            p = new spgemm_attention_plan_s();
            p->device = device;
            try {
                return build_plan(p, mask, backward != 0, slabs, (hipStream_t)stream);
            } catch (const ScratchError&) {
                // the bounds of the slabs fell short: once more without them
                SG_HIP(hipStreamSynchronize((hipStream_t)stream));
            }
        }
        return SPGEMM_ERR_INTERNAL;
    });
    if (rc != SPGEMM_OK) {
        if (p) (void)hipStreamSynchronize((hipStream_t)stream);
        delete p;
        return rc;
    }
    *out = p;
    return SPGEMM_OK;
}

SPGEMM_API void spgemm_attention_plan_destroy(spgemm_attention_plan p) {
    if (!p) return;
    (void)hipDeviceSynchronize();
    delete p;
}

SPGEMM_API int spgemm_attention_workspace(spgemm_attention_plan p,
                                          const spgemm_attention_desc* desc, int32_t backward,
                                          int64_t* bytes) {
    if (!p || !desc_valid(desc) || !bytes) return SPGEMM_ERR_INVALID_ARG;
    if (backward && !p->backward) return SPGEMM_ERR_NOT_READY;
    return guarded([&]() -> int {
        const AttnShape s = make_shape(desc);
        ForwardArgs f;
        BackwardArgs b;
        *bytes = backward ? carve_backward(p, s, nullptr, &b) : carve_forward(p, s, nullptr, &f);
        return SPGEMM_OK;
    });
}

SPGEMM_API int spgemm_attention_forward(spgemm_attention_plan p, const spgemm_attention_desc* desc,
                                        const spgemm_rows* q, const spgemm_rows* k,
                                        const spgemm_rows* v, const spgemm_rows* out, float* lse,
                                        void* workspace, int64_t workspace_bytes, void* stream) {
    if (!p || !desc_valid(desc)) return SPGEMM_ERR_INVALID_ARG;
    return guarded([&]() -> int {
        ForwardArgs a;
        a.s = make_shape(desc);
        a.side = row_side(p, &a.s);
        a.nrows = p->nrows;
        AttnRows kr, vr;
        if (!rows_valid(q, p->nrows, a.s.hq, desc, false, &a.q) ||
            !rows_valid(k, p->ncols, a.s.hkv, desc, false, &kr) ||
            !rows_valid(v, p->ncols, a.s.hkv, desc, false, &vr) ||
            !rows_valid(out, p->nrows, a.s.hq, desc, true, &a.out))
            return SPGEMM_ERR_INVALID_ARG;
        if (!make_gather(kr, p->ncols, 1, &a.k) || !make_gather(vr, p->ncols, 1, &a.v))
            return SPGEMM_ERR_OVERFLOW;
        if (!workspace_valid(workspace, workspace_bytes, carve_forward(p, a.s, workspace, &a)) ||
            !plan_here(p))
            return SPGEMM_ERR_INVALID_ARG;
        a.lse = lse;
        attention_forward(a, (hipStream_t)stream);
        return SPGEMM_OK;
    });
}

SPGEMM_API int spgemm_attention_backward(spgemm_attention_plan p,
                                         const spgemm_attention_desc* desc, const spgemm_rows* q,
                                         const spgemm_rows* k, const spgemm_rows* v,
                                         const spgemm_rows* out, const float* lse,
                                         const spgemm_rows* dout, const spgemm_rows* dq,
                                         const spgemm_rows* dk, const spgemm_rows* dv,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
    if (!p || !desc_valid(desc) || (!lse && p->nrows > 0)) return SPGEMM_ERR_INVALID_ARG;
    if (!p->backward) return SPGEMM_ERR_NOT_READY;
    return guarded([&]() -> int {
        BackwardArgs a;
        a.s = make_shape(desc);
        a.rows = row_side(p, &a.s);
        a.nrows = p->nrows;
        a.cols = col_side(p, a.s.hkv);
        a.ncols = p->ncols;
        if (!rows_valid(q, p->nrows, a.s.hq, desc, false, &a.q) ||
            !rows_valid(k, p->ncols, a.s.hkv, desc, false, &a.krow) ||
            !rows_valid(v, p->ncols, a.s.hkv, desc, false, &a.vrow) ||
            !rows_valid(out, p->nrows, a.s.hq, desc, false, &a.out) ||
            !rows_valid(dout, p->nrows, a.s.hq, desc, false, &a.dout) ||
            !rows_valid(dq, p->nrows, a.s.hq, desc, true, &a.dq) ||
            !rows_valid(dk, p->ncols, a.s.hkv, desc, true, &a.dk) ||
            !rows_valid(dv, p->ncols, a.s.hkv, desc, true, &a.dv))
            return SPGEMM_ERR_INVALID_ARG;
        if (!make_gather(a.krow, p->ncols, 1, &a.k) || !make_gather(a.vrow, p->ncols, 1, &a.v) ||
            !make_gather(a.q, p->nrows, a.s.hq, &a.gq) ||
            !make_gather(a.dout, p->nrows, a.s.hq, &a.gdout))
            return SPGEMM_ERR_OVERFLOW;
        if (!workspace_valid(workspace, workspace_bytes, carve_backward(p, a.s, workspace, &a)) ||
            !plan_here(p))
            return SPGEMM_ERR_INVALID_ARG;
        a.lse = lse;
        a.group_div = FastDiv((uint32_t)a.s.group);
        attention_backward(a, (hipStream_t)stream);
        return SPGEMM_OK;
    });
}

SPGEMM_API int spgemm_paged_attention_workspace(const spgemm_attention_desc* desc,
                                                const spgemm_paged_batch* batch, int64_t* bytes) {
    if (!desc_valid(desc) || !batch_sizes_valid(batch) || !bytes) return SPGEMM_ERR_INVALID_ARG;
    if (!batch_sizes_fit(batch, desc)) return SPGEMM_ERR_OVERFLOW;
    return guarded([&]() -> int {
        PagedArgs a;
        a.s = make_shape(desc);
        batch_sizes(batch, &a);
        *bytes = carve_paged(nullptr, &a);
        return SPGEMM_OK;
    });
}

SPGEMM_API int spgemm_paged_attention(const spgemm_attention_desc* desc, const spgemm_rows* q,
                                      const spgemm_paged_cache* cache,
                                      const spgemm_paged_batch* batch, const spgemm_rows* out,
                                      float* lse, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
    if (!desc_valid(desc) || !batch_sizes_valid(batch) || !cache) return SPGEMM_ERR_INVALID_ARG;
    const spgemm_csr* pg = batch->pages;
    if (pg->nnz < 0 || cache->npages < 0 || cache->page_size < 1 || pg->ncols != cache->npages)
        return SPGEMM_ERR_INVALID_ARG;
    if (!batch_sizes_fit(batch, desc) || pg->nnz > 0x7fffffffLL || cache->npages > 0x7fffffffLL ||
        cache->page_size > kMaxTokens)
        return SPGEMM_ERR_OVERFLOW;
    return guarded([&]() -> int {
        PagedArgs a;
        a.s = make_shape(desc);
        batch_sizes(batch, &a);
        if (!rows_valid(q, a.tokens, a.s.hq, desc, false, &a.q) ||
            !rows_valid(out, a.tokens, a.s.hq, desc, true, &a.out))
            return SPGEMM_ERR_INVALID_ARG;
        if (a.seqs == 0 || a.tokens == 0 || a.max_new == 0) return SPGEMM_OK;
        if (!pg->rowptr || (pg->nnz > 0 && !pg->col) || !batch->q_rowptr || !batch->lengths)
            return SPGEMM_ERR_INVALID_ARG;
        const int size = type_size(desc->type);
        const int64_t counts[2] = {cache->npages, cache->page_size};
        const int64_t ks[3] = {stride_bytes(cache->k_stride_page, counts[0], size),
                               stride_bytes(cache->k_stride_slot, counts[1], size),
                               stride_bytes(cache->k_stride_head, a.s.hkv, size)};
        const int64_t vs[3] = {stride_bytes(cache->v_stride_page, counts[0], size),
                               stride_bytes(cache->v_stride_slot, counts[1], size),
                               stride_bytes(cache->v_stride_head, a.s.hkv, size)};
        for (int i = 0; i < 3; ++i)
            if (ks[i] < 0 || vs[i] < 0) return SPGEMM_ERR_INVALID_ARG;
        a.k = static_cast<const char*>(cache->k);
        a.v = static_cast<const char*>(cache->v);
        if (cache->npages > 0 &&
            (!a.k || !a.v || reinterpret_cast<uintptr_t>(a.k) % 16 != 0 ||
             reinterpret_cast<uintptr_t>(a.v) % 16 != 0))
            return SPGEMM_ERR_INVALID_ARG;
        if (!gather_unit(ks, counts, 2, &a.k_shift) || !gather_unit(vs, counts, 2, &a.v_shift))
            return SPGEMM_ERR_OVERFLOW;
        a.k_page = (uint32_t)(ks[0] >> a.k_shift);
        a.k_slot = (uint32_t)(ks[1] >> a.k_shift);
        a.v_page = (uint32_t)(vs[0] >> a.v_shift);
        a.v_slot = (uint32_t)(vs[1] >> a.v_shift);
        a.k_head = ks[2];
        a.v_head = vs[2];
        a.npages = cache->npages;
        a.page_div = FastDiv((uint32_t)cache->page_size);
        a.group_div = FastDiv((uint32_t)a.s.group);
        a.room = pg->nnz;
        a.rowptr = pg->rowptr;
        a.col = pg->col;
        a.q_rowptr = batch->q_rowptr;
        a.lengths = batch->lengths;
        a.lse = lse;
        if (!workspace_valid(workspace, workspace_bytes, carve_paged(workspace, &a)))
            return SPGEMM_ERR_INVALID_ARG;
        paged_attention(a, (hipStream_t)stream);
        return SPGEMM_OK;
    });
}

}  // extern "C"
