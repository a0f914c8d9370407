// paged.cuh -- the cache in pages, and which of its keys a call reads.
//
// Key j of sequence b is row j % page_size of page table[b][j / page_size].
// Query token t of a sequence of L keys is at position p = L - Sq + t and sees
// the keys j <= p with j > p - window (window 0: all) or j < first.  So a call
// reads the keys [0, first) and [lo, L), lo = max(0, L - Sq + 1 - window): the
// union over the tokens.  It reads them in boxes of `box` rows of a page (box:
// the largest of 128, 64, 32, 16 that divides the page size, at most what the
// kernel takes), and lays the boxes that hold a read key end to end, whole:
// the sequence as the schedule and the tiles see it.  Its rows are numbered by
//     i < split:  position i            (boxes of the first tokens)
//     i >= split: position i + jump     (boxes from the one that holds lo)
// with jump = 0 where nothing is left out.  Rows that no token sees -- past L,
// and around the ends of the two ranges in their boxes -- are masked in S and
// zeroed in shared memory before P V, so whatever they hold (a page's old
// contents, NaN) reaches no result.  Boxes past the end are loaded with a page
// index outside the cache, which TMA fills with zeros; so is a table entry
// outside it, which is also flagged.
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "schedule.cuh"

namespace mla {

constexpr uint32_t kStatusPage = 4u;  // a block-table entry outside the cache's pages, or a token without a place

struct PagedArgs {
    const int32_t* seqlens;    // [B], or one length for all (len_stride 0)
    const int32_t* table;      // rows of page indices
    long long table_stride;    // 0: every sequence reads the same row
    int len_stride;
    int L_max, num_pages, page_size;
    int box, box_log2;         // rows per TMA box
    int Sq;                    // query tokens (positions count back from L)
    int window, first;         // window 0: no window
    int mask_rows;             // query rows per token
    int whole_slot;            // >= 0: a whole sequence also leaves a partial, in slot whole_slot + b; -1: none does
};

// One sequence as read: its length, and its rows as the tiles number them.
struct SeqView {
    int L;      // keys
    int rows;   // rows read (tiles cover these)
    int split, jump;
    int lo;     // row of the first key seen through the window (0: no window)
};

__device__ __forceinline__ SeqView view_of(const PagedArgs& a, int L) {
    SeqView v;
    v.L = L;
    v.rows = L;
    v.split = v.jump = v.lo = 0;
    if (a.window > 0) {
        const int lo = L - a.Sq + 1 - a.window;
        if (lo > 0) {
            const int split = ((a.first + a.box - 1) >> a.box_log2) << a.box_log2;
            const int at = (lo >> a.box_log2) << a.box_log2;
            v.lo = lo;
            if (at > split) {
                v.split = split;
                v.jump = at - split;
                v.rows = L - v.jump;
                v.lo = lo - v.jump;
            }
        }
    }
    return v;
}

__device__ __forceinline__ int paged_len(const PagedArgs& a, int b) {
    return clamp_len(__ldg(a.seqlens + b * a.len_stride), a.L_max, nullptr);
}

struct PagedLens {
    const PagedArgs* a;  // the kernel's own parameter
    __device__ __forceinline__ int operator()(int b) const { return view_of(*a, paged_len(*a, b)).rows; }
};

// Rows seen by one query token: [0, f) and [b0, b1).
struct RowRange {
    int f, b0, b1;
    __device__ __forceinline__ bool sees(int i) const { return i < f || (i >= b0 && i < b1); }
    // every row of [i, i + n) is seen
    __device__ __forceinline__ bool all(int i, int n) const { return i >= b0 && i + n <= b1; }
};

__device__ __forceinline__ RowRange token_rows(const PagedArgs& a, const SeqView& v, int t) {
    const int p = v.L - a.Sq + t;
    RowRange r;
    r.f = 0;
    r.b0 = 0;
    r.b1 = p + 1 - v.jump;
    if (a.window > 0) {
        r.f = a.first < p + 1 ? a.first : p + 1;
        const int lo = p + 1 - a.window;
        if (lo > 0) r.b0 = lo - v.jump > 0 ? lo - v.jump : 0;
    }
    return r;
}

// Row i of a sequence is seen by none of its tokens.
__device__ __forceinline__ bool unseen(const PagedArgs& a, const SeqView& v, int i) {
    return i >= v.rows || (i < v.lo && i >= a.first);
}
// Some row of tile t is seen by none: the tile's values are cleared there.
__device__ __forceinline__ bool tile_unseen(const PagedArgs& a, const SeqView& v, int t) {
    const int i = t * kTileKV;
    return i + kTileKV > v.rows || (i < v.lo && i + kTileKV > a.first);
}

// One lane's box in each of a partition's tiles, in order, one tile at a time
// (a lane holds row offset `off` of every tile).  The page index is the table's
// entry as it is: usable() turns it into a TMA coordinate, so that the entry's
// load is waited for only where it is used.
struct Box {
    int page, row;  // page: the table's entry; -1 where the tile has no such box
    bool some;
};

template <class Walker>
struct BoxStream {
    const PagedArgs& a;
    Walker w;
    Piece pc;
    SeqView v;
    int t, off;
    bool live;

    __device__ __forceinline__ BoxStream(const PagedArgs& args, const Walker& walker, int offset)
        : a(args), w(walker), t(0), off(offset) {
        live = w.next(pc);
        if (live) {
            t = pc.tile_lo;
            v = view_of(a, paged_len(a, pc.b));
        }
    }
    __device__ __forceinline__ Box next() {
        Box x;
        x.page = 0;
        x.row = 0;
        x.some = false;
        if (!live) return x;
        const int i = t * kTileKV + off;
        if (i < v.rows) {
            const int pos = i < v.split ? i : i + v.jump;
            const int e = pos / a.page_size;
            x.page = __ldg(a.table + pc.b * a.table_stride + e);
            x.row = pos - e * a.page_size;
            x.some = true;
        }
        if (++t == pc.tile_hi) {
            live = w.next(pc);
            if (live) {
                t = pc.tile_lo;
                v = view_of(a, paged_len(a, pc.b));
            }
        }
        return x;
    }
};

// TMA page coordinate of a box: its page, or one outside the cache (zeros).
__device__ __forceinline__ int usable(const PagedArgs& a, const Box& x, uint32_t* status) {
    if (x.some && (x.page < 0 || x.page >= a.num_pages)) atomicOr(status, kStatusPage);
    return x.some && x.page >= 0 && x.page < a.num_pages ? x.page : a.num_pages;
}

// How a kernel's KV rows are found.  ContigKv: rows of one [B, L_max, ...]
// tensor; PagedKv: as above.
struct ContigKv {
    static constexpr bool kPaged = false;
    struct Args {};
    using Lens = SeqLens;
};
struct PagedKv {
    static constexpr bool kPaged = true;
    using Args = PagedArgs;
    using Lens = PagedLens;
};

template <class A>
__device__ __forceinline__ SeqLens make_lens(const A& a, const ContigKv::Args&) {
    return SeqLens{a.seqlens, a.L_max};
}
template <class A>
__device__ __forceinline__ PagedLens make_lens(const A&, const PagedArgs& pa) {
    return PagedLens{&pa};
}

// Masks one kv row's scores in the transposed kernels: x[j] is the score of
// query row first_row + j (`per` rows a token, tokens up to last_tok; columns
// past them are padding) at row kv_row of the tile that starts at row0.
template <int G>
__device__ __forceinline__ void mask_columns(const PagedArgs& a, const SeqView& v, float (&x)[G], int row0, int kv_row,
                                             int first_row, int per, int last_tok) {
    int tok = first_row / per, rem = first_row - tok * per;
    const RowRange first = token_rows(a, v, tok);
    const int last = (first_row + G - 1) / per;
    // a tile that every token sees whole needs no mask
    if (first.all(row0, kTileKV) && token_rows(a, v, last < last_tok ? last : last_tok).all(row0, kTileKV)) return;
    bool sees = first.sees(kv_row);
#pragma unroll
    for (int j = 0; j < G; ++j) {
        if (!sees) x[j] = -INFINITY;
        if (++rem == per) {
            rem = 0;
            sees = token_rows(a, v, ++tok).sees(kv_row);
        }
    }
}

// Clears the kBytes (64 or 128) at p, 16 at a time, starting at `first` so that
// the lanes of a warp that clear neighbouring rows use different banks.
template <int kBytes>
__device__ __forceinline__ void clear_row(uint8_t* p, int first) {
#pragma unroll
    for (int c = 0; c < kBytes / 16; ++c)
        *reinterpret_cast<uint4*>(p + (((c + first) & (kBytes / 16 - 1)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace mla
