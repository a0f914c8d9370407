// kernel_combine.cuh -- split-KV combine (log-sum-exp merge of partials).
//
// For a sequence whose KV tiles were cut across k > 1 partitions, partition
// pieces left (O_s / l_s, lse_s) in fp32.  The merged result is
//     lse = ln sum_s exp(lse_s),      out = sum_s exp(lse_s - lse) * (O_s / l_s)
// which is exactly the softmax over the union of the pieces' keys.  A
// per-head attention sink (one more softmax term without a value) enters the
// merged lse only, once per row.  The pages
// do not describe splitting; this is the standard identity for merging
// softmax-normalised partial results.  Sequences that were not cut were
// finished by the main kernel and are skipped; empty sequences (L = 0) are
// written here as out = 0, lse = -inf (or the head's sink logit).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"
#include "schedule.cuh"

namespace mla {

struct CombineArgs {
    const int32_t* seqlens;
    int B;
    int R;
    int L_max;
    int P;
    __nv_bfloat16* out;
    float* lse;
    const float* part_o;
    const float* part_lse;
    const float* sinks;  // [H] per-head attention-sink logits (natural-log units), or null
    int H;
    int split_tiles;     // 0: balanced schedule; > 0: batch-invariant chunks of this many tiles
};

// Grid (B, Y): CTA (b, y) owns sequence b's query rows [y*RY, (y+1)*RY) with
// RY = ceil(R / Y); its 8 warps take one row each at a time.  Warp 0 reads the
// lengths once (schedule and b's unit offset in one pass), so a sequence that
// was not cut costs its CTAs one scan and nothing else; Y is chosen by the
// host so that about two CTAs per SM share the merging of cut sequences.
// Within a row the kernel is bound by the latency of the partials it reads, so
// each lane keeps up to 4 partials x 4 float4 in flight, requested before the
// merged lse is known, instead of walking the partials one after another.
constexpr int kCombineThreads = 256;
constexpr int kCombineWarps = kCombineThreads / 32;

// CTAs per sequence along y: enough to give about two CTAs per SM when many
// rows must be merged, never more than one per 8 rows.
inline int combine_grid_y(int B, int R, int num_sms) {
    const int max_y = (R + kCombineWarps - 1) / kCombineWarps;
    int y = (2 * num_sms) / B;
    if (y < 1) y = 1;
    return y < max_y ? y : max_y;
}

// DV: value width (512 for MLA, 128 for MHA); a lane owns DV / 128 float4 columns.
// CV: where the lengths come from (paged.cuh); in a paged run a row may have
// seen no key of any piece: it gets out = 0 and lse = -inf (or its sink).
// kNarrow: a warp takes 128 columns of a row with 16 partials in flight, instead
// of the whole row with 4: for few rows of many pieces, where rows alone leave
// warps without work.
template <int DV = kDv, class CV = ContigKv, bool kNarrow = false>
__global__ void __launch_bounds__(kCombineThreads, 2)
    mla_decode_combine_kernel(const CombineArgs args, const __grid_constant__ typename CV::Args pa) {
    static_assert(DV == 512 || DV == 128, "value width");
    constexpr int NC = kNarrow ? DV / 128 : 1;  // column groups of a row
    constexpr int NV4 = DV / 128 / NC;          // float4 columns per lane
    constexpr int KB = kNarrow ? 16 : 4;        // partials in flight
    // weights a lane keeps, one for every 32 pieces: 5 are those of as many pieces
    // as a plan makes by itself (reading a weight again for each piece beyond the
    // 32nd, one sequence of 78 pieces takes 27 instead of 22 us; where pieces are
    // few, looking for them costs 0.3 us)
    constexpr int kHeld = kNarrow ? 5 : 1;
    __shared__ int s_split;
    __shared__ long long s_acc, s_tot;
    const int b = blockIdx.x;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // the schedule the main kernel used for these lengths, its unit count and
    // the flat unit offset of sequence b (units: tiles, or S-tile chunks)
    if (warp == 0) {
        const ScheduleScan sc = schedule_scan_warp(make_lens(args, pa), args.B, args.P, args.split_tiles, b);
        if (lane == 0) {
            s_split = sc.S;
            s_acc = sc.acc_at;
            s_tot = sc.units;
        }
    }
    __syncthreads();
    // launched as a programmatic dependent of the main kernel: the scan above
    // reads only the lengths; partials and outputs wait for the main grid
    ptx::wait_prior_grid();
    const int S = s_split;
    const long long acc = s_acc, tot = s_tot;
    // this CTA's (row, column group) units
    const int units = args.R * NC;
    const int units_per = (units + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
    const int u_lo = static_cast<int>(blockIdx.y) * units_per;
    const int u_hi = u_lo + units_per < units ? u_lo + units_per : units;
    const int L = make_lens(args, pa)(b);
    const long long n = num_units(L, S);
    if (n == 0) {
        for (int u = u_lo + warp; u < u_hi; u += kCombineWarps) {
            if (NC > 1 && u % NC != 0) continue;
            const int r = u / NC;
            const size_t orow = static_cast<size_t>(b) * args.R + r;
            // a per-head sink is one more softmax term without a value (-inf: none)
            const float sink = args.sinks ? args.sinks[r % args.H] : -INFINITY;
            uint4* dst = reinterpret_cast<uint4*>(args.out + orow * DV);  // DV / 8 x 16 bytes
            for (int i = lane; i < DV / 8; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
            if (lane == 0) args.lse[orow] = sink;  // nothing to attend to: the sink alone
        }
        return;
    }
    int k, p0 = 0;
    if (S > 0) {
        // chunk schedule: chunk i of b is in slot acc + i
        if (n == 1) return;  // one chunk: finished by the main kernel
        k = static_cast<int>(n);
    } else {
        const long long T = (tot + args.P - 1) / args.P;
        p0 = static_cast<int>(acc / T);
        const int p1 = static_cast<int>((acc + n - 1) / T);
        if (p0 == p1) return;  // finished by the main kernel
        k = p1 - p0 + 1;
    }
    // slot of the i-th piece: the first partition's piece continues after it
    // (2 p0 + 1), every later piece started before its partition (2 p)
    auto slot_of = [&](int i) {
        if (S > 0) return static_cast<int>(acc) + i;
        return (i == 0) ? 2 * p0 + 1 : 2 * (p0 + i);
    };

    for (int u = u_lo + warp; u < u_hi; u += kCombineWarps) {
        const int r = u / NC, col = (u % NC) * 32 + lane;  // first float4 column of the lane
        const size_t orow = static_cast<size_t>(b) * args.R + r;
        const float sink = args.sinks ? args.sinks[r % args.H] : -INFINITY;
        auto prow_of = [&](int i) { return static_cast<size_t>(slot_of(i)) * args.R + r; };
        // the first (up to) KB partial rows are requested before the lse values
        // are reduced, so a row cut into at most KB pieces costs one round trip
        float4 x[KB][NV4];
        auto load_batch = [&](int i0) {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (i0 + j < k) {
                    const float4* src = reinterpret_cast<const float4*>(args.part_o + prow_of(i0 + j) * DV);
#pragma unroll
                    for (int v = 0; v < NV4; ++v) x[j][v] = __ldcs(src + col + 32 * v);
                }
            }
        };
        load_batch(0);
        // merged lse: lane i holds pieces i, i + 32, ... (those beyond 32 kHeld folded in by a loop)
        float my_w[kHeld];
        float m = -INFINITY;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            my_w[h] = lane + 32 * h < k ? args.part_lse[prow_of(lane + 32 * h)] : -INFINITY;
            m = fmaxf(m, my_w[h]);
        }
        for (int i = lane + 32 * kHeld; i < k; i += 32) m = fmaxf(m, args.part_lse[prow_of(i)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = fmaxf(m, sink);
        if (CV::kPaged && m == -INFINITY) m = 0.f;
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            my_w[h] = lane + 32 * h < k ? expf(my_w[h] - m) : 0.f;
            sum += my_w[h];
        }
        for (int i = lane + 32 * kHeld; i < k; i += 32) sum += expf(args.part_lse[prow_of(i)] - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum += expf(sink - m);
        const float lse_all = m + logf(sum);
        const float inv = (CV::kPaged && sum == 0.f) ? 0.f : 1.f / sum;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) my_w[h] *= inv;  // weights of the lane's pieces: exp(lse_i - lse)

        // out = sum_i exp(lse_i - lse) * (O_i / l_i); lane owns float4 columns col + 32 v
        float4 acc_o[NV4];
#pragma unroll
        for (int v = 0; v < NV4; ++v) acc_o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < k; i0 += KB) {
            if (i0 > 0) load_batch(i0);
            float w_at = my_w[0];  // pieces [i0, i0 + KB) are in one group of 32
#pragma unroll
            for (int h = 1; h < kHeld; ++h) w_at = i0 >= 32 * h ? my_w[h] : w_at;
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                const int i = i0 + j;
                if (i < k) {
                    const float w = i < 32 * kHeld ? __shfl_sync(0xffffffffu, w_at, i & 31)
                                                   : expf(args.part_lse[prow_of(i)] - m) * inv;
#pragma unroll
                    for (int v = 0; v < NV4; ++v) {
                        acc_o[v].x += w * x[j][v].x;
                        acc_o[v].y += w * x[j][v].y;
                        acc_o[v].z += w * x[j][v].z;
                        acc_o[v].w += w * x[j][v].w;
                    }
                }
            }
        }
        __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(args.out + orow * DV);
#pragma unroll
        for (int v = 0; v < NV4; ++v) {
            const int e0 = (col + 32 * v) * 4;  // first column of acc_o[v]
            const __nv_bfloat162 lo = __floats2bfloat162_rn(acc_o[v].x, acc_o[v].y);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(acc_o[v].z, acc_o[v].w);
            uint2 pk;
            pk.x = *reinterpret_cast<const uint32_t*>(&lo);
            pk.y = *reinterpret_cast<const uint32_t*>(&hi);
            *reinterpret_cast<uint2*>(dst + e0 / 2) = pk;
        }
        if (lane == 0 && (NC == 1 || col == 0)) args.lse[orow] = lse_all;
    }
}

// Shared prefix.  A row's keys are the prefix's (pieces of the 128-row group
// that holds the row, rows of all sequences end to end) and its sequence's own;
// every piece of either left a partial, and this merges them.  Pieces of a
// group and of a sequence are found as the main kernels' schedules cut them.
struct PrefixCombineArgs {
    int B, R, H;
    int P_own, P_pre;           // partitions of the two main launches
    int groups;                 // 128-row groups, the last one perhaps not full
    __nv_bfloat16* out;
    float* lse;
    const float* own_o;         // [2 P_own + B, R, 512]
    const float* own_lse;
    const float* pre_o;         // [2 P_pre + groups, 128, 512]
    const float* pre_lse;
    const float* sinks;
};

__global__ void __launch_bounds__(kCombineThreads, 2)
    mla_prefix_combine_kernel(const PrefixCombineArgs args, const __grid_constant__ PagedArgs own,
                              const __grid_constant__ PagedArgs pre) {
    constexpr int NV4 = kDv / 128;
    constexpr int kHeld = 3;  // weights a lane keeps, one for every 32 pieces
    __shared__ int s_split;
    __shared__ long long s_acc, s_tot;
    const int b = blockIdx.x;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (warp == 0) {
        const ScheduleScan sc = schedule_scan_warp(PagedLens{&own}, args.B, args.P_own, 0, b);
        if (lane == 0) {
            s_split = sc.S;
            s_acc = sc.acc_at;
            s_tot = sc.units;
        }
    }
    __syncthreads();
    ptx::wait_prior_grid();
    // this sequence's own pieces: k_own of them from slot s0 on, then every second one
    const long long n = num_units(PagedLens{&own}(b), s_split);
    int k_own = 0, own_p0 = 0;
    bool own_whole = true;
    if (n > 0) {
        k_own = 1;
        if (s_split == 0) {
            const long long T = (s_tot + args.P_own - 1) / args.P_own;
            own_p0 = static_cast<int>(s_acc / T);
            k_own = static_cast<int>((s_acc + n - 1) / T) - own_p0 + 1;
            own_whole = (k_own == 1);
        }
    }
    // the prefix: every group has the same tiles
    const long long n_pre = num_tiles(PagedLens{&pre}(0));
    const bool pre_one = pick_schedule(n_pre * args.groups, n_pre, args.groups, args.P_pre, pre.cut_tiles) > 0;
    const long long T_pre = n_pre > 0 ? (n_pre * args.groups + args.P_pre - 1) / args.P_pre : 1;

    const int rows_per = (args.R + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
    const int r_lo = static_cast<int>(blockIdx.y) * rows_per;
    const int r_hi = r_lo + rows_per < args.R ? r_lo + rows_per : args.R;
    for (int r = r_lo + warp; r < r_hi; r += kCombineWarps) {
        const long long orow = static_cast<long long>(b) * args.R + r;
        const long long grp = orow >> 7;
        int k_pre = 0, pre_p0 = 0;
        bool pre_whole = true;
        if (n_pre > 0) {
            k_pre = 1;
            if (!pre_one) {
                pre_p0 = static_cast<int>(grp * n_pre / T_pre);
                k_pre = static_cast<int>((grp * n_pre + n_pre - 1) / T_pre) - pre_p0 + 1;
                pre_whole = (k_pre == 1);
            }
        }
        const int k = k_own + k_pre;
        const float sink = args.sinks ? args.sinks[r % args.H] : -INFINITY;
        // partial row of piece i: the sequence's pieces, then the group's
        auto prow_of = [&](int i) -> size_t {
            if (i < k_own) {
                const long long s = own_whole ? 2LL * args.P_own + b : (i == 0 ? 2 * own_p0 + 1 : 2 * (own_p0 + i));
                return static_cast<size_t>(s * args.R + r);
            }
            const int j = i - k_own;
            const long long s = pre_whole ? 2LL * args.P_pre + grp : (j == 0 ? 2 * pre_p0 + 1 : 2 * (pre_p0 + j));
            return static_cast<size_t>(s * 128 + (orow & 127));
        };
        auto lse_of = [&](int i) { return (i < k_own ? args.own_lse : args.pre_lse)[prow_of(i)]; };
        float4 x[4][NV4];
        auto load_batch = [&](int i0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (i0 + j < k) {
                    const float4* src = reinterpret_cast<const float4*>(
                        (i0 + j < k_own ? args.own_o : args.pre_o) + prow_of(i0 + j) * kDv);
#pragma unroll
                    for (int v = 0; v < NV4; ++v) x[j][v] = __ldcs(src + lane + 32 * v);
                }
            }
        };
        load_batch(0);
        float my_w[kHeld];
        float m = -INFINITY;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            my_w[h] = lane + 32 * h < k ? lse_of(lane + 32 * h) : -INFINITY;
            m = fmaxf(m, my_w[h]);
        }
        for (int i = lane + 32 * kHeld; i < k; i += 32) m = fmaxf(m, lse_of(i));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = fmaxf(m, sink);
        if (m == -INFINITY) m = 0.f;  // nothing to see and no sink: out = 0, lse = -inf
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) {
            my_w[h] = lane + 32 * h < k ? expf(my_w[h] - m) : 0.f;
            sum += my_w[h];
        }
        for (int i = lane + 32 * kHeld; i < k; i += 32) sum += expf(lse_of(i) - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum += expf(sink - m);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int h = 0; h < kHeld; ++h) my_w[h] *= inv;
        float4 acc_o[NV4];
#pragma unroll
        for (int v = 0; v < NV4; ++v) acc_o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < k; i0 += 4) {
            if (i0 > 0) load_batch(i0);
            float w_at = my_w[0];
#pragma unroll
            for (int h = 1; h < kHeld; ++h) w_at = i0 >= 32 * h ? my_w[h] : w_at;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j;
                if (i < k) {
                    const float w = i < 32 * kHeld ? __shfl_sync(0xffffffffu, w_at, i & 31)
                                                   : expf(lse_of(i) - m) * inv;
#pragma unroll
                    for (int v = 0; v < NV4; ++v) {
                        acc_o[v].x += w * x[j][v].x;
                        acc_o[v].y += w * x[j][v].y;
                        acc_o[v].z += w * x[j][v].z;
                        acc_o[v].w += w * x[j][v].w;
                    }
                }
            }
        }
        __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(args.out + orow * kDv);
#pragma unroll
        for (int v = 0; v < NV4; ++v) {
            const int e0 = (lane + 32 * v) * 4;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(acc_o[v].x, acc_o[v].y);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(acc_o[v].z, acc_o[v].w);
            uint2 pk;
            pk.x = *reinterpret_cast<const uint32_t*>(&lo);
            pk.y = *reinterpret_cast<const uint32_t*>(&hi);
            *reinterpret_cast<uint2*>(dst + e0 / 2) = pk;
        }
        if (lane == 0) args.lse[orow] = m + logf(sum);
    }
}

}  // namespace mla
