// kernel_append.cuh -- appending new tokens to a paged cache with the
// position rotation applied on the way.
//
// Token i of the flattened new tokens belongs to the sequence b with
// cu[b] <= i < cu[b+1] and sits at position p = L_b - n_b + (i - cu[b])
// (L_b: the sequence's length with its new tokens, n_b = cu[b+1] - cu[b]).  Its
// row goes to page table[b][p / page_size], row p % page_size; the row's
// rotated columns, and the token's query rows, turn by the angles of p:
//     (x0, x1) -> (x0 c - x1 s, x1 c + x0 s),   c, s = cos_sin[p]
// with pairs (2i, 2i+1) (interleaved) or (i, i + n/2).  Behind a shared prefix of
// P keys the row's place is the same and the angles are those of P + p.  All of
// it is fp32, rounded once when it is written (products and sums each rounded, no
// fused multiply-add, so the result is the one elementary operations give).
//
// Every input is read once and every output written once, and a token needs only
// its own rows: 8 to 10 us at HBM's rate for prompts of 8000 to 10000 tokens.  What
// bounds it is the chain of loads to a token's place, walked by 2 to 3 waves of
// warps one after the other: 14 to 16 us with inputs out of L2, 9 to 11 with them in
// it.  A token's work is in tasks of about 2 KB -- its cache
// row, or 8 (128 wide) / 16 (64 wide) head rows -- dealt to `parts` warps: one
// where there are tokens enough to fill the GPU (which sequence, its length, its
// page and its angles, a chain of loads, are then found once), more where there
// are few.  A warp issues its first task's loads before it looks for the token's
// place, and each further task's before it writes the one at hand.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "paged.cuh"
#include "schedule.cuh"

namespace mla {


struct AppendArgs {
    int B, T;
    int per_seq;                // tokens of every sequence when cu is null
    const int32_t* cu;          // [B + 1] or null
    const int32_t* seqlens;     // [B], with the new tokens
    const int32_t* prefix_len;  // keys in front of every sequence, or null
    const int32_t* table;
    long long table_stride;
    int table_width, num_pages, page_size;
    const float* cos_sin;       // [num_positions, rot]: rot / 2 cosines, rot / 2 sines
    int num_positions, rot;
    uint32_t* status;           // or null
    // head rows: key rows (MHA), value rows (MHA), query rows; element strides
    const __nv_bfloat16* k;     // MLA: latent [T, 512]
    long long k_token, k_head;
    const __nv_bfloat16* v;     // MLA: k_rope [T, 64]
    long long v_token, v_head;
    const __nv_bfloat16* q_in;  // or null
    long long qi_token, qi_head;
    __nv_bfloat16* q_out;
    long long qo_token, qo_head;
    int H, Hkv;
    void* k_pages;              // MLA: the cache's rows of 576
    __nv_bfloat16* v_pages;
    float kv_scale;             // E4M3 cache
    float kv_inv;               // 1 / kv_scale rounded, or 0 where that or its products could leave fp32's range
};

constexpr int kAppendThreads = 128;
constexpr int kAppendRowBytes = 2048;  // head-row bytes of one task

// Sequence and place of token i, and the position whose angles it turns by; place
// -1: the token is in no sequence (padding), or its place is negative or that
// position outside [0, num_positions) (flagged).  Warp-cooperative: each round of the search narrows the bounds 32-fold (the lanes read
// evenly spaced ones, and the last at most i opens the next range), and the last
// round reads the lengths with them, so that a token's chain of loads is one
// shorter.
__device__ __forceinline__ void place_token(const AppendArgs& a, int i, int lane, int& b, int& pos, int& angle) {
    long long next, L;
    int prefix = a.prefix_len ? __ldg(a.prefix_len) : 0;
    if (a.cu) {
        int lo = 0, n = a.B + 1;  // the answer is in [lo, lo + n)
        while (n > 32) {
            const int step = (n + 31) >> 5;
            const int at = lane * step;
            const unsigned m = __ballot_sync(0xffffffffu, at < n && __ldg(a.cu + lo + at) <= i);
            if (m == 0) break;
            const int last = 31 - __clz(m);
            lo += last * step;
            n = n - last * step < step ? n - last * step : step;
        }
        const int at = lo + lane;
        int opens = 0, closes = 0, len = 0;
        if (lane < n && at < a.B) {
            opens = __ldg(a.cu + at);
            closes = __ldg(a.cu + at + 1);
            len = __ldg(a.seqlens + at);
        }
        const unsigned m = __ballot_sync(0xffffffffu, lane < n && at < a.B && opens <= i);
        const int last = m == 0 ? 0 : 31 - __clz(m);
        b = lo + last;
        next = __shfl_sync(0xffffffffu, closes, last);
        L = __shfl_sync(0xffffffffu, len, last);
        if (m == 0 || i >= next) {
            pos = -1;
            return;
        }
    } else {
        b = i / a.per_seq;
        next = static_cast<long long>(b + 1) * a.per_seq;
        L = __ldg(a.seqlens + b);
    }
    const long long p = L - next + i;
    pos = -1;
    bool good = prefix >= 0;  // (a negative one counts as 0, as in the decode)
    if (!good) prefix = 0;
    if (p >= 0 && p + prefix < a.num_positions) {
        pos = static_cast<int>(p);
        angle = pos + prefix;
    } else {
        good = false;
    }
    if (!good && a.status && lane == 0) atomicOr(a.status, kStatusSeqlen);
}

// Row of the cache for position pos of sequence b, or -1 (flagged).
__device__ __forceinline__ long long cache_row(const AppendArgs& a, int b, int pos, int lane) {
    const int e = pos / a.page_size;
    int page = -1;
    if (e < a.table_width) page = __ldg(a.table + b * a.table_stride + e);
    if (page < 0 || page >= a.num_pages) {
        if (a.status && lane == 0) atomicOr(a.status, kStatusPage);
        return -1;
    }
    return static_cast<long long>(page) * a.page_size + (pos - e * a.page_size);
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// x / scale from the reciprocal inv: the product and one correction by its exact
// remainder, which gives the correctly rounded quotient (Markstein, IBM J. Res.
// Dev. 34, 1990).  A division of each of 576 columns took 2 of 12.7 us for 8168
// tokens.  Beyond what E4M3 holds the product itself will do (infinities, NaN).
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
    const float q = x * inv;
    return fabsf(q) < 1024.f ? fmaf(fmaf(-q, scale, x), inv, q) : q;
}

// Eight E4M3 codes of x / scale, saturated at +-448 (round to nearest even).
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float scale, float inv) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = inv != 0.f ? make_float2(quotient(x[2 * i], scale, inv), quotient(x[2 * i + 1], scale, inv))
                                    : make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
        const uint32_t c = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
        w[i >> 1] |= (c & 0xFFFFu) << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

// The angles of this lane's columns col .. col + 7 (col < rot).
template <bool kInterleaved>
struct Angles {
    float c[kInterleaved ? 4 : 8], s[kInterleaved ? 4 : 8];
    __device__ __forceinline__ void load(const float* row, int col, int rot) {
        const int half = rot >> 1;
        const int at = kInterleaved ? (col >> 1) : (col < half ? col : col - half);
#pragma unroll
        for (int j = 0; j < (kInterleaved ? 4 : 8); j += 4) {
            *reinterpret_cast<float4*>(c + j) = __ldg(reinterpret_cast<const float4*>(row + at + j));
            *reinterpret_cast<float4*>(s + j) = __ldg(reinterpret_cast<const float4*>(row + half + at + j));
        }
    }
};

// Turns this lane's 8 columns.  Half-split pairs sit in the lane `rot / 16`
// away (all lanes of the warp take part in the exchange).
template <bool kInterleaved>
__device__ __forceinline__ void turn8(float (&x)[8], const Angles<kInterleaved>& a, int col, int rot, int lane) {
    if constexpr (kInterleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = x[2 * j], w = x[2 * j + 1];
            x[2 * j] = __fsub_rn(__fmul_rn(u, a.c[j]), __fmul_rn(w, a.s[j]));
            x[2 * j + 1] = __fadd_rn(__fmul_rn(w, a.c[j]), __fmul_rn(u, a.s[j]));
        }
    } else {
        const bool low = col < (rot >> 1);
        const int partner = low ? lane + rot / 16 : lane - rot / 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float y = __shfl_sync(0xffffffffu, x[j], partner & 31);
            x[j] = low ? __fsub_rn(__fmul_rn(x[j], a.c[j]), __fmul_rn(y, a.s[j]))
                       : __fadd_rn(__fmul_rn(x[j], a.c[j]), __fmul_rn(y, a.s[j]));
        }
    }
}

// Heads [h0, h0 + n) of one token, W columns each: read, turned (columns below
// rot), written.  n <= kAppendRowBytes / (2 W), so all loads are in flight at once.
template <int W>
struct HeadRows {
    static constexpr int kLanes = W / 8;                                      // lanes per row
    static constexpr int kRows = 32 / kLanes;                                 // rows at a time
    static constexpr int kSteps = kAppendRowBytes / (2 * W) / kRows;          // 4
    static constexpr int kHeads = kRows * kSteps;
    uint4 raw[kSteps];
    __device__ __forceinline__ void load(const __nv_bfloat16* src, long long head_stride, int n, int lane) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int h = i * kRows + lane / kLanes;
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (h < n) raw[i] = *reinterpret_cast<const uint4*>(src + h * head_stride + (lane % kLanes) * 8);
        }
    }
    template <bool kInterleaved>
    __device__ __forceinline__ void turn(const Angles<kInterleaved>& ang, int rot, int lane) {
        const int col = (lane % kLanes) * 8;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            float x[8];
            unpack8(raw[i], x);
            turn8<kInterleaved>(x, ang, col, rot, lane);
            if (col < rot) raw[i] = pack8(x);
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16* dst, long long head_stride, int n, int lane) const {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int h = i * kRows + lane / kLanes;
            if (h < n) *reinterpret_cast<uint4*>(dst + h * head_stride + (lane % kLanes) * 8) = raw[i];
        }
    }
};

// The token and part of this warp: grid (T / warps a block, parts).
__device__ __forceinline__ long long token_of_warp() {
    return static_cast<long long>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
}

// Latent cache: a token's task 0 is its row [latent 512 | turned k_rope 64], the
// others 16 of its query heads' rope columns each.
template <bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads) mla_cache_append_kernel(const AppendArgs a) {
    using R = HeadRows<64>;
    const int lane = threadIdx.x & 31, parts = gridDim.y;
    const long long token = token_of_warp();
    if (token >= a.T) return;
    const int i = static_cast<int>(token);
    const int tasks = 1 + (a.H + R::kHeads - 1) / R::kHeads;
    const bool row_here = blockIdx.y == 0;
    int task = row_here ? parts : blockIdx.y;  // the first task of heads
    const __nv_bfloat16* q_in = a.q_in + i * a.qi_token;
    auto heads = [&](int t) { return a.H - (t - 1) * R::kHeads < R::kHeads ? a.H - (t - 1) * R::kHeads : R::kHeads; };
    auto load = [&](R& rows, int t) { rows.load(q_in + (t - 1) * R::kHeads * a.qi_head, a.qi_head, heads(t), lane); };
    R rows;
    if (task < tasks) load(rows, task);
    const __nv_bfloat16* latent = a.k + i * a.k_token;
    // bf16: columns 8 lane, 256 + 8 lane (rows of 512 bytes a step); E4M3: 16 lane .. 16 lane + 15 (16 bytes of codes)
    const int c0 = kFp8 ? 16 * lane : 8 * lane, c1 = kFp8 ? 16 * lane + 8 : 256 + 8 * lane;
    const int col = (lane & 7) * 8;
    uint4 r0, r1, raw = make_uint4(0u, 0u, 0u, 0u);
    if (row_here) {
        r0 = *reinterpret_cast<const uint4*>(latent + c0);
        r1 = *reinterpret_cast<const uint4*>(latent + c1);
        if (lane < 8) raw = *reinterpret_cast<const uint4*>(a.v + i * a.v_token + col);
    }
    int b, pos, angle;
    place_token(a, i, lane, b, pos, angle);
    if (pos < 0) return;
    Angles<kInterleaved> ang;
    ang.load(a.cos_sin + static_cast<long long>(angle) * a.rot, col, a.rot);
    const long long row = row_here ? cache_row(a, b, pos, lane) : -1;
    if (row >= 0) {
        float x[8];
        unpack8(raw, x);
        turn8<kInterleaved>(x, ang, col, a.rot, lane);
        if constexpr (kFp8) {
            uint8_t* dst = static_cast<uint8_t*>(a.k_pages) + row * kDqk;
            float y[8], z[8];
            unpack8(r0, y);
            unpack8(r1, z);
            const uint2 lo = quantise8(y, a.kv_scale, a.kv_inv), hi = quantise8(z, a.kv_scale, a.kv_inv);
            *reinterpret_cast<uint4*>(dst + c0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            if (lane < 8) *reinterpret_cast<uint2*>(dst + kDv + col) = quantise8(x, a.kv_scale, a.kv_inv);
        } else {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.k_pages) + row * kDqk;
            *reinterpret_cast<uint4*>(dst + c0) = r0;
            *reinterpret_cast<uint4*>(dst + c1) = r1;
            if (lane < 8) *reinterpret_cast<uint4*>(dst + kDv + col) = pack8(x);
        }
    }
    __nv_bfloat16* q_out = a.q_out + i * a.qo_token;
    for (; task < tasks; task += parts) {
        R next;
        if (task + parts < tasks) load(next, task + parts);
        rows.template turn<kInterleaved>(ang, a.rot, lane);
        rows.store(q_out + (task - 1) * R::kHeads * a.qo_head, a.qo_head, heads(task), lane);
        rows = next;
    }
}

// Keys and values of grouped kv heads, 128 wide: a token's tasks are its key
// heads (turned), its value heads (copied) and its query heads, 8 at a time.
template <bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads) mha_cache_append_kernel(const AppendArgs a) {
    using R = HeadRows<128>;
    const int lane = threadIdx.x & 31, parts = gridDim.y;
    const long long token = token_of_warp();
    if (token >= a.T) return;
    const int i = static_cast<int>(token);
    const int kv_tasks = (a.Hkv + R::kHeads - 1) / R::kHeads;
    const int tasks = 2 * kv_tasks + (a.H + R::kHeads - 1) / R::kHeads;
    struct Task {
        int kind, h0, n;  // kind 0: keys, 1: values, 2: queries
    };
    auto task_at = [&](int t) {
        Task k;
        k.kind = t < kv_tasks ? 0 : t < 2 * kv_tasks ? 1 : 2;
        k.h0 = (t - k.kind * kv_tasks) * R::kHeads;
        const int heads = k.kind == 2 ? a.H : a.Hkv;
        k.n = heads - k.h0 < R::kHeads ? heads - k.h0 : R::kHeads;
        return k;
    };
    auto load = [&](R& rows, const Task& k) {
        const __nv_bfloat16* from = k.kind == 0   ? a.k + i * a.k_token
                                    : k.kind == 1 ? a.v + i * a.v_token
                                                  : a.q_in + i * a.qi_token;
        const long long step = k.kind == 0 ? a.k_head : k.kind == 1 ? a.v_head : a.qi_head;
        rows.load(from + k.h0 * step, step, k.n, lane);
    };
    int t = blockIdx.y;
    Task at = task_at(t);
    R rows;
    load(rows, at);
    int b, pos, angle;
    place_token(a, i, lane, b, pos, angle);
    if (pos < 0) return;
    const int col = (lane % R::kLanes) * 8;
    Angles<kInterleaved> ang;
    if (col < a.rot) ang.load(a.cos_sin + static_cast<long long>(angle) * a.rot, col, a.rot);
    const long long row = t < 2 * kv_tasks ? cache_row(a, b, pos, lane) : -1;
    while (true) {
        R next;
        Task then;
        const bool more = t + parts < tasks;
        if (more) {
            then = task_at(t + parts);
            load(next, then);
        }
        if (at.kind != 1) rows.template turn<kInterleaved>(ang, a.rot, lane);
        if (at.kind == 2) {
            rows.store(a.q_out + i * a.qo_token + at.h0 * a.qo_head, a.qo_head, at.n, lane);
        } else if (row >= 0) {
            __nv_bfloat16* pages = at.kind == 1 ? a.v_pages : static_cast<__nv_bfloat16*>(a.k_pages);
            rows.store(pages + (row * a.Hkv + at.h0) * 128, 128, at.n, lane);
        }
        if (!more) return;
        t += parts;
        at = then;
        rows = next;
    }
}

}  // namespace mla
