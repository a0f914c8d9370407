// schedule.cuh -- split-KV work distribution shared by the main and combine
// kernels (device side; computed from the lengths that live on the device, so
// a run needs no host synchronisation and can be captured in a CUDA graph).
//
// The KV tiles (kTileKV rows each) of all sequences are laid end to end:
// sequence b owns tiles [acc_b, acc_b + n_b) of a flat index space of N_t
// tiles.  The space is cut into P equal contiguous ranges of T = ceil(N_t/P)
// tiles ("partitions"); partition p is processed by one CTA (or CTA pair) per
// query-row group.  A sequence that falls inside one partition is finished by
// that CTA; a sequence cut by partition boundaries leaves one fp32 partial
// (O / l and its log-sum-exp) per piece, merged by the combine kernel.
//
// Partial slots: partition p owns slots 2p and 2p+1.  The piece of sequence b
// in partition p uses slot 2p if b started before p, else slot 2p+1 (b starts
// in p and continues after it).  Both can occur in one partition, for two
// different sequences; a sequence that both starts before and ends after p is
// p's only sequence and uses 2p.
//
// Batch-invariant schedule (S > 0 tiles).  Where a sequence is cut above
// depends on every other sequence of the batch, and so do the rounding of
// its partials and of their merge.  With S > 0 the unit of work is instead a
// chunk of S tiles of one sequence (its last chunk shorter): chunk k of
// sequence b covers tiles [kS, min(kS + S, n_b)), is always a piece of its
// own, and a sequence of u_b > 1 chunks writes chunk k to slot acc_b + k
// (acc_b = chunks of the sequences before b).  The flat list of chunks is cut
// into P equal ranges as before; only which CTA computes a chunk depends on
// the batch, not what it computes, so a sequence's output is bitwise the same
// in any batch.  The same units serve runs whose S is chosen for them (below).
#pragma once

#include <cstdint>

namespace mla {

constexpr int kTileKV = 128;       // kv rows per pipeline tile
constexpr int kDqk = 576;          // 512 latent + 64 rope
constexpr int kDv = 512;
constexpr int kChunk = 64;         // columns per 128-byte swizzled chunk
constexpr int kNumChunks = kDqk / kChunk;  // 9

// status word bits (workspace header, word 0)
constexpr uint32_t kStatusTimeout = 1u;
constexpr uint32_t kStatusSeqlen = 2u;

__device__ __forceinline__ int clamp_len(int L, int L_max, uint32_t* status) {
    if (L < 0 || L > L_max) {
        if (status) atomicOr(status, kStatusSeqlen);
        L = L < 0 ? 0 : L_max;
    }
    return L;
}

__device__ __forceinline__ int num_tiles(int L) { return (L + kTileKV - 1) / kTileKV; }

// schedule units of a sequence of L keys: its tiles (S = 0) or its S-tile chunks
__device__ __forceinline__ long long num_units(int L, int S) {
    const int n = num_tiles(L);
    return S > 0 ? (n + S - 1) / S : n;
}

// Sum over a warp of values below 2^42, by the warp's 32-bit reductions (ten
// 64-bit shuffles a sum took most of the scan's time).
__device__ __forceinline__ long long warp_sum(long long v) {
    const unsigned lo = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v) & 0xffffu);
    const unsigned hi = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v >> 16));
    return (static_cast<long long>(hi) << 16) + lo;
}

// Schedule actually used for a run (warp-cooperative; every CTA and the
// combine kernel reach the same answer from the same lengths).  A plan's
// split_tiles > 0 (batch-invariant) is kept.  Otherwise the balanced schedule
// is used, except when a whole sequence per partition is expected to finish
// sooner: cutting a sequence costs about kCutTiles tiles of time (an extra
// epilogue that stalls the pipeline, the fp32 partials and their merge), and
// a balanced partition holds up to two cut pieces.  So when every non-empty
// sequence fits its own partition, the sequences keep at least half of the
// partitions busy, and the longest sequence is no longer than the balanced
// share plus two cuts, each sequence is one piece (returned as a chunk size
// covering the longest sequence).
constexpr int kCutTiles = 5;

// Where the schedule's functions take a sequence's number of keys from (a
// callable b -> keys, with the cost of a cut in tiles, and whether a run may be cut
// evenly).  SeqLens: an array of
// lengths on the device.
struct SeqLens {
    const int32_t* seqlens;
    int L_max;
    __device__ __forceinline__ int operator()(int b) const { return clamp_len(__ldg(seqlens + b), L_max, nullptr); }
    __device__ __forceinline__ int cut() const { return kCutTiles; }
    __device__ __forceinline__ bool even() const { return false; }
};

struct ScheduleScan {
    int S;             // chunk size in tiles of this run's schedule (0: balanced over tiles)
    long long units;   // schedule units over all sequences (tiles, or chunks)
    long long acc_at;  // units of the sequences before sequence `b_at` (0 when b_at < 0)
};

// The chunk size of a run whose plan leaves the choice (0: balanced).
__device__ __forceinline__ int pick_schedule(long long total, long long n_max, long long nonempty, int P, int cut) {
    if (n_max == 0 || nonempty > P || 2 * nonempty < P) return 0;
    const long long T = (total + P - 1) / P;
    return n_max <= T + 2 * cut ? static_cast<int>(n_max) : 0;
}

// One pass over the lengths (warp-cooperative): the schedule of this run, its
// number of units and, for b_at >= 0, the flat unit offset of sequence b_at.
// Every quantity whose unit depends on the schedule is accumulated for each
// candidate (tiles; chunks of the plan's size; non-empty sequences, the unit of
// the one-piece-per-sequence schedule), so one pass serves all three.
template <class Lens>
__device__ inline ScheduleScan schedule_scan_warp(const Lens& lens, int B, int P, int plan_split, int b_at = -1) {
    const int lane = threadIdx.x & 31;
    long long total = 0, chunks = 0, at_tiles = 0, at_chunks = 0;
    int n_max = 0, nonempty = 0, at_nonempty = 0;
    for (int b = lane; b < B; b += 32) {
        const int L = lens(b);
        const int n = num_tiles(L);
        const long long c = plan_split > 0 ? num_units(L, plan_split) : 0;
        total += n;
        n_max = n > n_max ? n : n_max;
        nonempty += (n > 0);
        chunks += c;
        if (b < b_at) {
            at_tiles += n;
            at_nonempty += (n > 0);
            at_chunks += c;
        }
    }
    if (plan_split > 0) return {plan_split, warp_sum(chunks), b_at > 0 ? warp_sum(at_chunks) : 0};
    total = warp_sum(total);
    nonempty = __reduce_add_sync(0xffffffffu, nonempty);
    n_max = __reduce_max_sync(0xffffffffu, n_max);
    const int S = pick_schedule(total, n_max, nonempty, P, lens.cut());
    if (S > 0) return {S, nonempty, b_at > 0 ? __reduce_add_sync(0xffffffffu, at_nonempty) : 0};
    // A balanced partition mostly holds two pieces.  Where chunks of a size less
    // than a cut above the balanced share leave one to a partition, those take
    // their place (29 sequences of 128 rows over E4M3 pages, L = 1800: 52 -> 39 us).  Half a
    // chunk a sequence is lost on average: no search where that is too much.
    const long long T = (total + P - 1) / P;
    if (lens.even() && T > 1 && total + nonempty * (T + lens.cut()) / 2 <= P * (T + lens.cut())) {
        const int first = static_cast<int>(T);
#pragma unroll 1
        for (int s = first; s < first + lens.cut(); ++s) {
            int units = 0, at = 0;
#pragma unroll 1
            for (int b = lane; b < B; b += 32) {
                const int u = static_cast<int>(num_units(lens(b), s));
                units += u;
                if (b < b_at) at += u;
            }
            units = __reduce_add_sync(0xffffffffu, units);
            if (units <= P) return {s, units, b_at > 0 ? __reduce_add_sync(0xffffffffu, at) : 0};
        }
    }
    return {0, total, b_at > 0 ? warp_sum(at_tiles) : 0};
}

// Locate the first sequence overlapping flat unit `start` (warp-cooperative).
template <class Lens>
__device__ inline void locate_warp(const Lens& lens, int B, int S, long long start, int* b_out, long long* acc_out) {
    const int lane = threadIdx.x & 31;
    long long acc = 0;
    for (int base = 0; base < B; base += 32) {
        const int b = base + lane;
        const int n = (b < B) ? static_cast<int>(num_units(lens(b), S)) : 0;  // < 2^18
        const int sum = __reduce_add_sync(0xffffffffu, n);
        if (acc + sum > start) {
            // inclusive prefix within the warp
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            // the first sequence with n > 0 whose range [acc + incl - n, acc + incl) reaches past start
            const unsigned m = __ballot_sync(0xffffffffu, n > 0 && acc + incl > start);
            const int src = __ffs(m) - 1;
            *b_out = base + src;
            *acc_out = acc + __shfl_sync(0xffffffffu, incl - n, src);
            return;
        }
        acc += sum;
    }
    *b_out = B;
    *acc_out = acc;
}

struct Piece {
    int b;          // sequence
    int L;          // its (clamped) length
    int tile_lo;    // first tile (sequence-local index)
    int tile_hi;    // one past the last tile
    int slot;       // partial slot, or -1 when the piece is the whole sequence
};

// Sequential walker over the pieces of one partition; every role of a CTA
// runs its own copy and sees the same sequence of pieces.
template <class Lens>
struct PieceWalkerOf {
    Lens lens;
    int B, p;
    int S;                 // 0: balanced schedule over tiles; > 0: chunks of S tiles
    long long start, end;  // flat unit range of this partition
    int b;                 // next sequence to look at
    long long acc;         // its flat offset (in units)
    long long k;           // S > 0: next chunk of sequence b

    __device__ bool next(Piece& out) {
        if (S > 0) return next_chunk(out);
        while (b < B && acc < end) {
            const int L = lens(b);
            const long long n = num_tiles(L);
            const long long lo = acc > start ? acc : start;
            const long long hi = (acc + n) < end ? (acc + n) : end;
            const int cur = b;
            const long long acc_cur = acc;
            ++b;
            acc += n;
            if (hi <= lo) continue;
            out.b = cur;
            out.L = L;
            out.tile_lo = static_cast<int>(lo - acc_cur);
            out.tile_hi = static_cast<int>(hi - acc_cur);
            const bool starts_before = acc_cur < start;
            const bool continues_after = acc_cur + n > end;
            if (!starts_before && !continues_after) out.slot = -1;
            else out.slot = starts_before ? 2 * p : 2 * p + 1;
            return true;
        }
        return false;
    }

    // batch-invariant schedule: one S-tile chunk per piece
    __device__ bool next_chunk(Piece& out) {
        while (b < B && acc + k < end) {
            const int L = lens(b);
            const int n = num_tiles(L);  // < 2^18, and so is S: 32-bit division
            const int u = (n + S - 1) / S;
            if (acc + k < start) k = start - acc;
            if (k >= u) {
                acc += u;
                ++b;
                k = 0;
                continue;
            }
            out.b = b;
            out.L = L;
            out.tile_lo = static_cast<int>(k * S);
            out.tile_hi = static_cast<int>((k + 1) * S < n ? (k + 1) * S : n);
            out.slot = (u == 1) ? -1 : static_cast<int>(acc + k);
            ++k;
            return true;
        }
        return false;
    }
};
using PieceWalker = PieceWalkerOf<SeqLens>;

}  // namespace mla
