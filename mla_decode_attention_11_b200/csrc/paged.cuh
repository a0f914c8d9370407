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
// with jump = 0 where nothing is left out.  Behind a shared prefix of P keys the
// rows below split = P rounded up to a box are the prefix's, found in its own
// table, and the sequence's own keys follow with jump = -split.  Rows that no
// token sees -- past L, and around the ends of the two ranges in their boxes -- are
// masked in S and zeroed in shared memory before P V, so whatever they hold (a
// page's old contents, NaN) reaches no result.  Boxes past the end are loaded with a page
// index outside the cache, which TMA fills with zeros; so is a table entry
// outside it, which is also flagged.
#pragma once

#include <cuda.h>
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
    uint32_t page_mul;         // position / page_size = position * page_mul >> page_shift, for positions below 2^25
    int page_shift;
    int box, box_log2;         // rows per TMA box
    int cut_tiles;             // the schedule's cost of a cut (schedule.cuh)
    int Sq;                    // query tokens (positions count back from L)
    int window, first;         // no window: 2^30, which no length reaches, and 0
    int split;                 // first rounded up to a box
    int heads_log2;            // query rows per token (latent caches: H, a power of two)
    // a shared prefix in front of every sequence's own keys, or null
    const int32_t* prefix_table;
    const int32_t* prefix_len;  // one length
    int prefix_max;
    int whole_slot;            // >= 0: a whole sequence also leaves a partial, in slot whole_slot + b; -1: none does
    CUtensorMap prefetch;      // E4M3 pages: boxes of `box` rows x all columns, for prefetches into L2
};

// One sequence as read: its length, and its rows as the tiles number them.
struct SeqView {
    int L;      // keys (own keys behind a prefix)
    int rows;   // rows read (tiles cover these)
    int split, jump;
    int f, lo;  // rows [f, lo) are seen by no token
};

__device__ __forceinline__ SeqView view_of(const PagedArgs& a, int L) {
    SeqView v;
    v.L = L;
    if (a.prefix_table) {
        const int P = clamp_len(__ldg(a.prefix_len), a.prefix_max, nullptr);
        v.f = P;
        v.split = v.lo = ((P + a.box - 1) >> a.box_log2) << a.box_log2;
        v.jump = -v.split;
        v.rows = L > 0 ? v.split + L : P;
    } else {
        const int lo = L - a.Sq + 1 - a.window, left_out = (lo & -a.box) - a.split;
        v.f = a.first;
        v.split = a.split;
        v.jump = left_out > 0 ? left_out : 0;
        v.rows = L - v.jump;
        v.lo = (lo > 0 ? lo : 0) - v.jump;
    }
    return v;
}

__device__ __forceinline__ int paged_len(const PagedArgs& a, int b) {
    return clamp_len(__ldg(a.seqlens + b * a.len_stride), a.L_max, nullptr);
}

struct PagedLens {
    const PagedArgs* a;  // the kernel's own parameter
    __device__ __forceinline__ int operator()(int b) const { return view_of(*a, paged_len(*a, b)).rows; }
    __device__ __forceinline__ int cut() const { return a->cut_tiles; }
    // (where whole sequences leave partials, the merge knows whole and balanced runs only)
    __device__ __forceinline__ bool even() const { return a->whole_slot < 0; }
};

// Rows seen by one query token: [0, f) and [b0, b1).
struct RowRange {
    int f, b0, b1;
    __device__ __forceinline__ bool sees(int i) const { return i < f || (i >= b0 && i < b1); }
    // every row of [i, i + n) is seen
    __device__ __forceinline__ bool all(int i, int n) const { return (i >= b0 && i + n <= b1) || i + n <= f; }
};

__device__ __forceinline__ RowRange token_rows(const PagedArgs& a, const SeqView& v, int t) {
    const int p = v.L - a.Sq + t;
    RowRange r;
    r.b1 = p + 1 - v.jump;
    if (a.prefix_table) {
        r.f = v.f;
        r.b0 = v.split;
    } else {
        r.f = a.first < p + 1 ? a.first : p + 1;
        r.b0 = r.b1 - a.window > 0 ? r.b1 - a.window : 0;
    }
    return r;
}

// Bits j of [0, 64) with lo <= j < hi.
__device__ __forceinline__ uint64_t bits_between(int lo, int hi) {
    const uint64_t below = hi >= 64 ? ~0ull : hi <= 0 ? 0ull : (1ull << hi) - 1;
    return lo >= 64 ? 0ull : lo <= 0 ? below : below & ~((1ull << lo) - 1);
}

// Rows to clear: those that no token sees in boxes that were loaded.  (Boxes past
// the sequence's end are zeros as TMA wrote them.)
__device__ __forceinline__ bool unseen(const PagedArgs& a, const SeqView& v, int i) {
    return (i >= v.rows && i < ((v.rows + a.box - 1) & -a.box)) || (i < v.lo && i >= v.f);
}
// Tile t has such rows.
__device__ __forceinline__ bool tile_unseen(const PagedArgs& a, const SeqView& v, int t) {
    const int i = t * kTileKV;
    return (i + kTileKV > v.rows && (v.rows & (a.box - 1))) || (i < v.lo && i + kTileKV > v.f);
}

// The boxes of a partition's tiles, found by a producer warp for the one of its
// threads that issues their loads.  A thread alone would wait for a table entry
// (and divide by the page size) before each tile; so the warp looks up 32 boxes
// at a time, a lane each, and leaves them in a list of 64 in shared memory:
// while that thread issues the tiles of one half, the entries of the next are on
// their way.  The thread is the one elect.sync names, so that the compiler knows
// TMA's operands to be one thread's.  Polling, arming and issuing with the whole
// warp instead (a box a lane) cost 23 % at 128 heads and 22 % over grouped kv heads
// even where a tile is one box or two.
// kMost: the most boxes of a tile.
template <class Walker, int kMost>
struct BoxList {
    static constexpr int kEntries = 64;
    const PagedArgs& a;
    int2* list;          // (page, row) of each box; page num_pages: outside the cache, TMA writes zeros
    Walker w;
    Piece pc;
    SeqView v;
    int t, lane, first_row, n_log2;
    int tiles, page, row;  // the batch being looked up: its tiles, this lane's box (page: the table's entry)
    bool some;

    // boxes of `rows` rows of every tile, from its row first_row on
    __device__ __forceinline__ BoxList(const PagedArgs& args, const Walker& walker, void* smem, int lane_, int first,
                                       int rows_log2)
        : a(args), list(static_cast<int2*>(smem)), w(walker), t(0), lane(lane_), first_row(first),
          n_log2(rows_log2 - args.box_log2) {
        pc.tile_hi = 0;  // no piece yet
    }

    // calls load(i, row, page) for each box i of a tile
    struct Boxes {
        int2 box[kMost];
        int count;
        template <class Load>
        __device__ __forceinline__ void each(Load load) const {
            // counts are powers of two: one test settles the usual one or two boxes
            load(0, box[0].y, box[0].x);
#pragma unroll
            for (int n = 1; n < kMost; n *= 2) {
                if (n >= count) return;
#pragma unroll
                for (int i = n; i < 2 * n; ++i) load(i, box[i].y, box[i].x);
            }
        }
    };
    __device__ __forceinline__ Boxes get(int tile) const {
        Boxes b;
        b.count = 1 << n_log2;
        const int2* from = list + ((tile << n_log2) & (kEntries - 1));
        b.box[0] = from[0];
#pragma unroll
        for (int n = 1; n < kMost; n *= 2)
            if (n < b.count)
#pragma unroll
                for (int i = n; i < 2 * n; ++i) b.box[i] = from[i];
        return b;
    }

    // All lanes call it; the elected one (always the same) calls
    // issue(tile, more) for each tile in order until it returns false.  more: the
    // next tile's boxes are known too.
    template <class Issue>
    __device__ __forceinline__ bool run(uint32_t* status, Issue issue) {
        // one copy of each step, and few instructions before the first load: at the
        // start of a kernel every line of code is fetched from L2 or beyond
        int done = 0, known = 0;
        bool ok = true;
        while (true) {
            look_up();
            // the last known tile waits for the next one to be known
            const int limit = tiles == 0 ? known : known - 1;
            if (ptx::elect_one())
                for (int i = done; ok && i < limit; ++i) ok = issue(i, i + 1 < known);
            done = limit > done ? limit : done;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || tiles == 0) return ok;
            publish(known, status);
            known += tiles;
        }
    }

    __device__ __forceinline__ void look_up() {
        tiles = 0;
        some = false;
        const int most = 32 >> n_log2, mine = lane >> n_log2;
        while (tiles < most) {
            if (t == pc.tile_hi) {
                if (!w.next(pc)) return;
                t = pc.tile_lo;
                v = view_of(a, paged_len(a, pc.b));
            }
            const int left = pc.tile_hi - t, take = left < most - tiles ? left : most - tiles;
            if (mine >= tiles && mine < tiles + take) {
                const int i = (t + mine - tiles) * kTileKV + first_row + ((lane & ((1 << n_log2) - 1)) << a.box_log2);
                if (i < v.rows) {
                    const int pos = i < v.split ? i : i + v.jump;
                    const int e = static_cast<int>(static_cast<uint64_t>(pos) * a.page_mul >> a.page_shift);
                    const bool shared = a.prefix_table && i < v.split;
                    page = __ldg((shared ? a.prefix_table : a.table + pc.b * a.table_stride) + e);
                    row = pos - e * a.page_size;
                    some = true;
                }
            }
            tiles += take;
            t += take;
        }
    }
    __device__ __forceinline__ void publish(int known, uint32_t* status) {
        const bool good = some && page >= 0 && page < a.num_pages;
        if (some && !good) atomicOr(status, kStatusPage);
        if (lane < (tiles << n_log2))
            list[((known << n_log2) + lane) & (kEntries - 1)] = make_int2(good ? page : a.num_pages, good ? row : 0);
        __syncwarp();
    }
};

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

// A row's reference maximum before it has seen a key, in place of -inf: then
// 2^(x - m) is 0 for its masked scores, and 2^(m - m_new) is 0, without a test.
constexpr float kNoKey = -3.0e38f;

// The columns of a transposed kernel's tile that do not see row kv_row: column
// j is row rem + j of token tok on (`per` rows a token; columns past the last
// token are padding).
__device__ __forceinline__ uint32_t hidden_columns(const PagedArgs& a, const SeqView& v, int columns, int tok, int rem,
                                                   int per, int kv_row) {
    uint32_t bits = 0;
#pragma unroll 1
    for (int j = -rem; j < columns; j += per, ++tok)
        if (!token_rows(a, v, tok).sees(kv_row)) bits |= static_cast<uint32_t>(bits_between(j, j + per));
    return bits;
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
