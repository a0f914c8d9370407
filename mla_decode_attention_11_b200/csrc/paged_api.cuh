// paged_api.cuh -- host side of the paged-cache entry points (plans, argument
// checks, tensor maps, launches).  Part of mla_decode.cu, which includes it
// after its own helpers.
#pragma once

#include "kernel_append.cuh"
#include "paged.cuh"

namespace {

constexpr int kMaxPageSize = 1 << 24;

// The largest box (rows of one TMA load) that divides the page size, at most
// `most`: 128 in the transposed kernel (a tile), 64 in the pair kernel (a CTA's
// keys of a tile).  Fewer, larger loads: one costs its issuing thread a few
// hundred cycles whatever it moves.
int page_box(int page_size, int most) {
    int box = most;
    while (page_size % box != 0) box /= 2;
    return box;
}

int box_log2(int box) { return box == 128 ? 7 : box == 64 ? 6 : box == 32 ? 5 : 4; }

mla_status check_page_args(int32_t page_size, int32_t window, int32_t first_tokens) {
    if (page_size < 1 || page_size > kMaxPageSize || window < 0 || first_tokens < 0 || first_tokens > (1 << 24))
        return MLA_ERR_INVALID_ARG;
    return page_size % 16 == 0 ? MLA_OK : MLA_ERR_UNSUPPORTED;
}

struct PrefixLayout {
    size_t pre_lse, pre_o, own_lse, own_o, total;
};

// Where whole sequences leave a partial too, a cut costs less than kCutTiles:
// 132 sequences of up to 16 tiles, 32 rows each, after a prefix of 16384 keys take
// 218 us uncut, 206 cut into equal shares.
constexpr int kPartialCutTiles = 2;

// shared prefix: slots of the prefix's pieces (two per partition, one per
// 128-row group) and of the sequences' own (two per partition, one per sequence)
PrefixLayout prefix_layout(const mla_plan& pl) {
    const size_t R = static_cast<size_t>(pl.Sq) * pl.H;
    const size_t pre = 128 * (2 * static_cast<size_t>(pl.prefix_partitions) + pl.prefix_groups);
    const size_t own = R * (2 * static_cast<size_t>(pl.num_partitions) + pl.B);
    PrefixLayout l;
    l.pre_lse = kHeaderBytes;
    l.own_lse = align_up(l.pre_lse + pre * sizeof(float), 256);
    l.pre_o = align_up(l.own_lse + own * sizeof(float), 256);
    l.own_o = align_up(l.pre_o + pre * mla::kDv * sizeof(float), 256);
    l.total = l.own_o + own * mla::kDv * sizeof(float);
    return l;
}

// Whether every sequence reads the prefix in front of its own keys, in one
// launch, or the prefix has a launch of its own for 128 rows of any sequences at
// a time.  With 128 rows a sequence both do the same products, and one launch
// balances them together and leaves no partial of a sequence that is not cut.
// With fewer, a sequence's own pass over the prefix takes NG / 148 of its tiles'
// time each, about 2.7 us a tile of a CTA, and the second launch and the partials
// some 20 us: the two are level at 8 tiles a CTA (64 sequences, 16 heads: 41 and
// 41 us; at 4 29 and 39, at 16 64 and 45).  The plan decides, by the longest prefix
// that it allows: a short one behind a plan for long ones takes the two launches.
bool prefix_in_front(const mla_plan& pl) {
    if (pl.kernel == MLA_KERNEL_PAIR) return true;
    const int64_t tiles = (static_cast<int64_t>(pl.prefix_max) + mla::kTileKV - 1) / mla::kTileKV;
    return tiles * pl.B * pl.num_groups <= 8 * static_cast<int64_t>(pl.num_sms);
}

// Latent pages [num_pages, page_size, 576]: boxes of `rows` rows x 64 columns x
// `chunks` adjacent 64-column chunks, chunk after chunk in shared memory
// (chunks = 1: a 3-D map {576, page_size, num_pages}).
bool encode_pages(EncodeTiledFn enc, CUtensorMap* m, const void* kv, int page_size, int num_pages, int rows,
                  int chunks) {
    return chunks == 1 ? encode_kv(enc, m, kv, page_size, num_pages, rows)
                       : encode_kv_chunks(enc, m, kv, page_size, num_pages, rows, chunks);
}

mla::PagedArgs paged_args(const mla_plan& pl, const int32_t* seqlens, const int32_t* table, int64_t table_stride,
                          int32_t num_pages, bool pair) {
    mla::PagedArgs a;
    std::memset(&a, 0, sizeof a);
    a.seqlens = seqlens;
    a.len_stride = 1;
    a.table = table;
    a.table_stride = table_stride;
    a.L_max = pl.L_max;
    a.num_pages = num_pages;
    a.page_size = pl.page_size;
    // positions n < 2^25: with 2^s >= page_size > 2^(s-1) and mul = ceil(2^(25+s) / page_size), n * (mul * page_size -
    // 2^(25+s)) < 2^25 * page_size <= 2^(25+s), so n * mul >> (25+s) is exact; mul < 2^27
    int s = 0;
    while ((1 << s) < pl.page_size) ++s;
    a.page_shift = 25 + s;
    a.page_mul = static_cast<uint32_t>(((1ull << a.page_shift) + pl.page_size - 1) / pl.page_size);
    a.box = page_box(pl.page_size, pair ? 64 : 128);
    a.box_log2 = box_log2(a.box);
    a.Sq = pl.Sq;
    const bool windowed = pl.window > 0 && pl.window < pl.L_max;  // one that no sequence fills leaves nothing out
    a.window = windowed ? pl.window : 1 << 30;
    a.first = !windowed ? 0 : pl.first_tokens < pl.L_max ? pl.first_tokens : pl.L_max;
    a.split = (a.first + a.box - 1) / a.box * a.box;
    while ((1 << a.heads_log2) < pl.H) ++a.heads_log2;
    a.whole_slot = -1;
    a.cut_tiles = mla::kCutTiles;
    return a;
}

void main_args(mla::MainArgs& a, const mla_plan& pl, const int32_t* seqlens, float softmax_scale, const float* sinks,
               void* out, float* lse, void* workspace, size_t lse_off, size_t o_off) {
    std::memset(&a, 0, sizeof a);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.seqlens = seqlens;
    a.B = pl.B;
    a.R = pl.Sq * pl.H;
    a.L_max = pl.L_max;
    a.P = pl.num_partitions;
    a.NG = pl.num_groups;
    a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634074);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.part_o = reinterpret_cast<float*>(ws + o_off);
    a.part_lse = reinterpret_cast<float*>(ws + lse_off);
    a.status = reinterpret_cast<uint32_t*>(ws);
    const unsigned long long tmo = g_timeout_ns.load();
    a.timeout_ns = tmo ? tmo : kDefaultTimeoutNs;
    a.stall_unit = g_stall_unit.load();
    a.prefetch_tiles = pl.l2_prefetch_tiles;
    a.sinks = sinks;
    a.H = pl.H;
    a.Sq = pl.Sq;
    a.Hkv = pl.Hkv;
    a.o_scale = 1.f;
}

// What every paged decode checks of its plan (but the plan's kind) and pointers.
mla_status check_paged(const mla_plan* plan, const void* q, const void* k, const void* v, int32_t num_pages,
                       const int32_t* table, int64_t table_stride, int32_t table_width, const int32_t* seqlens,
                       float softmax_scale, const float* sinks, const void* out, const float* lse) {
    if (!plan || !q || !k || !v || !table || !seqlens || !out || !lse) return MLA_ERR_INVALID_ARG;
    if (!std::isfinite(softmax_scale)) return MLA_ERR_INVALID_ARG;
    const mla_plan& pl = *plan;
    if (pl.B < 1 || pl.Sq < 1 || pl.H < 1 || pl.Hkv < 1 || pl.L_max < 1 || pl.num_partitions < 1 ||
        pl.num_partitions > 4096 || pl.num_groups < 1 || pl.split_tiles != 0 || pl.l2_prefetch_tiles < 0 ||
        pl.l2_prefetch_tiles > 16 || pl.page_size < 1 ||
        check_page_args(pl.page_size, pl.window, pl.first_tokens) != MLA_OK)
        return MLA_ERR_INVALID_ARG;
    if (num_pages < 1 || table_stride < 0 || table_width < 1 ||
        static_cast<int64_t>(table_width) * pl.page_size < pl.L_max)
        return MLA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(seqlens, 4) || !aligned(table, 4) || !aligned(sinks, 4))
        return MLA_ERR_ALIGNMENT;
    return MLA_OK;
}

bool mla_groups_ok(const mla_plan& pl) {
    const int R = pl.Sq * pl.H;
    if (pl.Hkv != 1 || pl.head_dim != mla::kDqk || pl.group_rows * pl.num_groups != R) return false;
    if (pl.kernel == MLA_KERNEL_PAIR) return pl.group_rows == 128;
    return pl.kernel == MLA_KERNEL_TRANSPOSED && (pl.group_rows == 16 || pl.group_rows == 32);
}

// The main kernel of an MLA plan over pages.
mla_status launch_mla_paged(EncodeTiledFn enc, const mla_plan& pl, const void* q, uint64_t q_rows, const void* kv,
                            const mla::MainArgs& a, const mla::PagedArgs& pa, uint64_t part_rows, cudaStream_t stream,
                             bool overlap = false) {
    CUtensorMap tm_q, tm_k, tm_v, tm_pf, tm_out, tm_part;
    if (pl.kernel == MLA_KERNEL_PAIR) {
        if (!encode_q_chunks(enc, &tm_q, q, q_rows) ||
            !encode_pages(enc, &tm_k, kv, pa.page_size, pa.num_pages, pa.box, 1) ||
            !encode_pages(enc, &tm_v, kv, pa.page_size, pa.num_pages, pa.box, 2) ||
            !encode_pages(enc, &tm_pf, kv, pa.page_size, pa.num_pages, pa.box, mla::kNumChunks) ||
            !encode_rows_store(enc, &tm_out, a.out, q_rows, false) ||
            !encode_rows_store(enc, &tm_part, a.part_o, part_rows, true))
            return MLA_ERR_CUDA;
        return launch_pair<mla::PagedKv>(pl, tm_q, tm_k, tm_v, tm_pf, tm_out, tm_part, a, pa, stream);
    }
    if (!encode_2d_bf16(enc, &tm_q, q, mla::kDqk, q_rows, mla::kChunk, pl.group_rows) ||
        !encode_pages(enc, &tm_k, kv, pa.page_size, pa.num_pages, pa.box, 1))
        return MLA_ERR_CUDA;
    return pl.group_rows == 16
               ? launch_transposed<16, mla::MlaShape, mla::PagedKv>(pl, tm_q, tm_k, tm_k, a, pa, stream, overlap)
               : launch_transposed<32, mla::MlaShape, mla::PagedKv>(pl, tm_q, tm_k, tm_k, a, pa, stream, overlap);
}

mla::CombineArgs combine_args(const mla::MainArgs& a) {
    mla::CombineArgs c;
    std::memset(&c, 0, sizeof c);
    c.seqlens = a.seqlens;
    c.B = a.B;
    c.R = a.R;
    c.L_max = a.L_max;
    c.P = a.P;
    c.out = a.out;
    c.lse = a.lse;
    c.part_o = a.part_o;
    c.part_lse = a.part_lse;
    c.sinks = a.sinks;
    c.H = a.H;
    return c;
}

dim3 combine_grid(const mla_plan& pl) {
    return dim3(static_cast<unsigned>(pl.B),
                static_cast<unsigned>(mla::combine_grid_y(pl.B, pl.Sq * pl.H, pl.num_sms)));
}

// The merge of a paged decode's pieces: narrow where a warp a row would leave
// half of the two CTAs an SM without work and a sequence has more pieces than the
// wide one has in flight (18 pieces: 20.9 -> 18.4 us a decode; 3: 13.4 -> 14.5).
template <int DV>
mla_status launch_paged_combine(const mla_plan& pl, const mla::MainArgs& a, const mla::PagedArgs& pa,
                                cudaStream_t stream) {
    const int R = pl.Sq * pl.H;
    const int64_t keys = static_cast<int64_t>(pl.prefix_max) +
                         (pa.window <= pl.L_max ? pa.split + pa.window + pl.Sq + 2 * pa.box : pl.L_max);
    const int64_t pieces = std::min<int64_t>((keys + mla::kTileKV - 1) / mla::kTileKV, pl.num_partitions / pl.B + 1);
    if (pieces <= 4 || static_cast<int64_t>(pl.B) * R > static_cast<int64_t>(pl.num_sms) * mla::kCombineWarps)
        return launch_dependent(mla::mla_decode_combine_kernel<DV, mla::PagedKv>, combine_grid(pl),
                                mla::kCombineThreads, stream, 0, combine_args(a), pa);
    const dim3 grid(static_cast<unsigned>(pl.B),
                    static_cast<unsigned>(mla::combine_grid_y(pl.B, R * (DV / 128), pl.num_sms)));
    return launch_dependent(mla::mla_decode_combine_kernel<DV, mla::PagedKv, true>, grid, mla::kCombineThreads, stream,
                            0, combine_args(a), pa);
}

struct Prefix {
    const int32_t *table, *len;
};

// One decode over latent pages whose plan and arguments have been checked, the
// workspace and the device excepted.
mla_status run_mla_paged(const mla_plan& pl, const void* q, const void* kv_pages, int32_t num_pages,
                         const Prefix* prefix, const int32_t* block_table, int64_t table_stride,
                         const int32_t* seqlens, float softmax_scale, const float* sinks, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream_) {
    const int R = pl.Sq * pl.H;
    const Layout lay = workspace_layout(num_slots(pl), R);
    if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
    mla_status st = check_run_device(pl);
    if (st != MLA_OK) return st;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return MLA_ERR_CUDA;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    mla::MainArgs a;
    main_args(a, pl, seqlens, softmax_scale, sinks, out, lse, workspace, lay.part_lse_off, lay.part_o_off);
    mla::PagedArgs pa = paged_args(pl, seqlens, block_table, table_stride, num_pages, pl.kernel == MLA_KERNEL_PAIR);
    if (prefix) {
        pa.prefix_table = prefix->table;
        pa.prefix_len = prefix->len;
        pa.prefix_max = pl.prefix_max;
    }
    st = launch_mla_paged(enc, pl, q, static_cast<uint64_t>(pl.B) * R, kv_pages, a, pa,
                          static_cast<uint64_t>(num_slots(pl)) * R, stream);
    if (st != MLA_OK) {
        cudaGetLastError();
        return st;
    }
    return launch_paged_combine<mla::kDv>(pl, a, pa, stream);
}

}  // namespace

extern "C" {

mla_status mla_decode_plan_paged(int32_t B, int32_t Sq, int32_t H, int32_t L_max, int32_t page_size, int32_t window,
                                 int32_t first_tokens, int32_t device, int32_t num_partitions_override,
                                 mla_plan* plan, size_t* workspace_bytes) {
    if (!plan) return MLA_ERR_INVALID_ARG;
    mla_plan p;
    mla_status st = mla_decode_plan_kernel(B, Sq, H, L_max, device, num_partitions_override, 0, &p, nullptr);
    if (st == MLA_OK) st = check_page_args(page_size, window, first_tokens);
    if (st != MLA_OK) return st;
    p.page_size = page_size;
    p.window = window;
    p.first_tokens = first_tokens;
    *plan = p;
    if (workspace_bytes) *workspace_bytes = p.workspace_bytes;
    return MLA_OK;
}

mla_status mla_decode_run_paged(const mla_plan* plan, const void* q, const void* kv_pages, int32_t num_pages,
                                const int32_t* block_table, int64_t table_stride, int32_t table_width,
                                const int32_t* seqlens, float softmax_scale, const float* sinks, void* out, float* lse,
                                void* workspace, size_t workspace_bytes, void* stream) {
    const mla_status st = check_paged(plan, q, kv_pages, kv_pages, num_pages, block_table, table_stride, table_width,
                                      seqlens, softmax_scale, sinks, out, lse);
    if (st != MLA_OK) return st;
    if (!mla_groups_ok(*plan) || plan->prefix_max != 0) return MLA_ERR_INVALID_ARG;
    return run_mla_paged(*plan, q, kv_pages, num_pages, nullptr, block_table, table_stride, seqlens, softmax_scale,
                         sinks, out, lse, workspace, workspace_bytes, stream);
}

mla_status mla_decode_plan_paged_fp8(int32_t B, int32_t Sq, int32_t H, int32_t L_max, int32_t page_size,
                                     int32_t window, int32_t first_tokens, int32_t device,
                                     int32_t num_partitions_override, mla_plan* plan, size_t* workspace_bytes) {
    if (!plan) return MLA_ERR_INVALID_ARG;
    mla_plan p;
    mla_status st = mla_decode_plan_fp8_kernel(B, Sq, H, L_max, device, num_partitions_override, 0, &p, nullptr);
    if (st == MLA_OK) st = check_page_args(page_size, window, first_tokens);
    if (st != MLA_OK) return st;
    if (p.kernel == MLA_KERNEL_FP8_PAIR) p.smem_bytes = PairFp8PagedC::kSmemBytes;
    p.page_size = page_size;
    p.window = window;
    p.first_tokens = first_tokens;
    *plan = p;
    if (workspace_bytes) *workspace_bytes = p.workspace_bytes;
    return MLA_OK;
}

mla_status mla_decode_run_paged_fp8(const mla_plan* plan, const void* q, const void* kv_pages, int32_t num_pages,
                                    float kv_scale, const int32_t* block_table, int64_t table_stride,
                                    int32_t table_width, const int32_t* seqlens, float softmax_scale,
                                    const float* sinks, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                    void* stream_) {
    mla_status st = check_paged(plan, q, kv_pages, kv_pages, num_pages, block_table, table_stride, table_width, seqlens,
                                softmax_scale, sinks, out, lse);
    if (st != MLA_OK) return st;
    const mla_plan& pl = *plan;
    const int R = pl.Sq * pl.H, G = pl.group_rows;
    const bool pair = pl.kernel == MLA_KERNEL_FP8_PAIR;
    if (!(pair ? G == 128 : pl.kernel == MLA_KERNEL_FP8_MMA && (G == 16 || G == 32)) ||
        pl.Hkv != 1 || pl.head_dim != mla::kDqk || G * pl.num_groups != R || pl.prefix_max != 0 ||
        !(std::isfinite(kv_scale) && kv_scale > 0.f))
        return MLA_ERR_INVALID_ARG;
    const Layout lay = workspace_layout(num_slots(pl), R);
    if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
    st = check_run_device(pl);
    if (st != MLA_OK) return st;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return MLA_ERR_CUDA;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    mla::MainArgs a;
    main_args(a, pl, seqlens, softmax_scale, sinks, out, lse, workspace, lay.part_lse_off, lay.part_o_off);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * kv_scale * 1.4426950408889634074);
    a.o_scale = kv_scale;
    mla::PagedArgs pa = paged_args(pl, seqlens, block_table, table_stride, num_pages, pair);
    if (pair) {
        CUtensorMap tm_k, tm_v, tm_pf, tm_out, tm_part;
        if (!encode_kv_fp8(enc, &tm_k, kv_pages, pl.page_size, num_pages, pa.box) ||
            !encode_kv_fp8_chunks(enc, &tm_v, kv_pages, pl.page_size, num_pages, pa.box, 2) ||
            !encode_kv_fp8_chunks(enc, &tm_pf, kv_pages, pl.page_size, num_pages, pa.box, mla::kNumChunks) ||
            !encode_rows_store(enc, &tm_out, out, static_cast<uint64_t>(pl.B) * R, false) ||
            !encode_rows_store(enc, &tm_part, a.part_o, static_cast<uint64_t>(num_slots(pl)) * R, true))
            return MLA_ERR_CUDA;
        st = launch_pair_fp8<mla::PagedKv>(pl, tm_k, tm_v, tm_pf, tm_out, tm_part, a, pa, stream);
        if (st != MLA_OK) {
            cudaGetLastError();
            return st;
        }
        return launch_paged_combine<mla::kDv>(pl, a, pa, stream);
    }
    CUtensorMap tm_kv;
    if (!encode_kv_fp8(enc, &tm_kv, kv_pages, pl.page_size, num_pages, pa.box) ||
        !encode_kv_fp8_chunks(enc, &pa.prefetch, kv_pages, pl.page_size, num_pages, pa.box, mla::kNumChunks))
        return MLA_ERR_CUDA;
    st = (G == 16) ? launch_fp8mma<16, mla::PagedKv>(pl, tm_kv, a, pa, stream)
                   : launch_fp8mma<32, mla::PagedKv>(pl, tm_kv, a, pa, stream);
    if (st != MLA_OK) {
        cudaGetLastError();
        return st;
    }
    return launch_paged_combine<mla::kDv>(pl, a, pa, stream);
}

mla_status mha_decode_plan_paged(int32_t B, int32_t Sq, int32_t H, int32_t Hkv, int32_t L_max, int32_t page_size,
                                 int32_t window, int32_t first_tokens, int32_t device,
                                 int32_t num_partitions_override, mla_plan* plan, size_t* workspace_bytes) {
    if (!plan) return MLA_ERR_INVALID_ARG;
    mla_plan p;
    mla_status st = mha_decode_plan(B, Sq, H, Hkv, L_max, device, num_partitions_override, &p, nullptr);
    if (st == MLA_OK) st = check_page_args(page_size, window, first_tokens);
    if (st != MLA_OK) return st;
    p.page_size = page_size;
    p.window = window;
    p.first_tokens = first_tokens;
    *plan = p;
    if (workspace_bytes) *workspace_bytes = p.workspace_bytes;
    return MLA_OK;
}

mla_status mha_decode_run_paged(const mla_plan* plan, const void* q, const void* k_pages, const void* v_pages,
                                int32_t num_pages, const int32_t* block_table, int64_t table_stride,
                                int32_t table_width, const int32_t* seqlens, float softmax_scale, const float* sinks,
                                void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream_) {
    mla_status st = check_paged(plan, q, k_pages, v_pages, num_pages, block_table, table_stride, table_width, seqlens,
                                softmax_scale, sinks, out, lse);
    if (st != MLA_OK) return st;
    const mla_plan& pl = *plan;
    const int G = pl.group_rows;
    if (pl.kernel != MLA_KERNEL_MHA || pl.H % pl.Hkv != 0 || pl.num_groups != pl.Hkv || pl.head_dim != kMhaD ||
        (G != 16 && G != 32) || pl.Sq * (pl.H / pl.Hkv) > G || pl.prefix_max != 0)
        return MLA_ERR_INVALID_ARG;
    const int R = pl.Sq * pl.H, gq = pl.H / pl.Hkv;
    const Layout lay = workspace_layout(num_slots(pl), R, kMhaD);
    if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
    st = check_run_device(pl);
    if (st != MLA_OK) return st;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return MLA_ERR_CUDA;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    mla::MainArgs a;
    main_args(a, pl, seqlens, softmax_scale, sinks, out, lse, workspace, lay.part_lse_off, lay.part_o_off);
    const mla::PagedArgs pa = paged_args(pl, seqlens, block_table, table_stride, num_pages, false);
    CUtensorMap tm_q, tm_k, tm_v;
    const uint64_t dq[4] = {static_cast<uint64_t>(kMhaD), static_cast<uint64_t>(pl.H), static_cast<uint64_t>(pl.Sq),
                            static_cast<uint64_t>(pl.B)};
    const uint32_t bq[4] = {static_cast<uint32_t>(mla::kChunk), static_cast<uint32_t>(gq),
                            static_cast<uint32_t>(pl.Sq), 1u};
    const uint64_t dk[4] = {static_cast<uint64_t>(kMhaD), static_cast<uint64_t>(pl.Hkv),
                            static_cast<uint64_t>(pl.page_size), static_cast<uint64_t>(num_pages)};
    const uint32_t bk[4] = {static_cast<uint32_t>(mla::kChunk), 1u, static_cast<uint32_t>(pa.box), 1u};
    if (!encode_4d_bf16(enc, &tm_q, q, dq, bq) || !encode_4d_bf16(enc, &tm_k, k_pages, dk, bk) ||
        !encode_4d_bf16(enc, &tm_v, v_pages, dk, bk))
        return MLA_ERR_CUDA;
    st = (G == 16) ? launch_transposed<16, mla::MhaShape, mla::PagedKv>(pl, tm_q, tm_k, tm_v, a, pa, stream)
                   : launch_transposed<32, mla::MhaShape, mla::PagedKv>(pl, tm_q, tm_k, tm_v, a, pa, stream);
    if (st != MLA_OK) {
        cudaGetLastError();
        return st;
    }
    return launch_paged_combine<kMhaD>(pl, a, pa, stream);
}

mla_status mla_decode_plan_prefix(int32_t B, int32_t Sq, int32_t H, int32_t L_max, int32_t prefix_max,
                                  int32_t page_size, int32_t device, int32_t num_partitions_override, mla_plan* plan,
                                  size_t* workspace_bytes) {
    if (!plan || prefix_max < 1 || prefix_max > (1 << 24)) return MLA_ERR_INVALID_ARG;
    mla_plan p;
    mla_status st = mla_decode_plan_kernel(B, Sq, H, L_max, device, num_partitions_override, 0, &p, nullptr);
    if (st == MLA_OK) st = check_page_args(page_size, 0, 0);
    if (st != MLA_OK) return st;
    p.page_size = page_size;
    p.prefix_max = prefix_max;
    if (!prefix_in_front(p)) {
        p.prefix_groups = static_cast<int32_t>((static_cast<int64_t>(B) * Sq * H + 127) / 128);
        int P = num_partitions_override > 0 ? num_partitions_override : p.num_sms / 2;  // one CTA pair each
        if (P < 1) P = 1;
        p.prefix_partitions = P > 4096 ? 4096 : P;
        p.workspace_bytes = prefix_layout(p).total;
    }
    *plan = p;
    if (workspace_bytes) *workspace_bytes = p.workspace_bytes;
    return MLA_OK;
}

mla_status mla_decode_run_prefix(const mla_plan* plan, const void* q, const void* kv_pages, int32_t num_pages,
                                 const int32_t* prefix_table, int32_t prefix_width, const int32_t* prefix_len,
                                 const int32_t* block_table, int64_t table_stride, int32_t table_width,
                                 const int32_t* seqlens, float softmax_scale, const float* sinks, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream_) {
    mla_status st = check_paged(plan, q, kv_pages, kv_pages, num_pages, block_table, table_stride, table_width, seqlens,
                                softmax_scale, sinks, out, lse);
    if (st != MLA_OK) return st;
    const mla_plan& pl = *plan;
    const int R = pl.Sq * pl.H;
    if (!prefix_table || !prefix_len || !mla_groups_ok(pl) || pl.window != 0 || pl.prefix_max < 1 ||
        pl.prefix_max > (1 << 24) || prefix_width < 1 ||
        static_cast<int64_t>(prefix_width) * pl.page_size < pl.prefix_max)
        return MLA_ERR_INVALID_ARG;
    if (!aligned(prefix_table, 4) || !aligned(prefix_len, 4)) return MLA_ERR_ALIGNMENT;
    if (pl.prefix_partitions == 0) {
        const Prefix prefix = {prefix_table, prefix_len};
        return run_mla_paged(pl, q, kv_pages, num_pages, &prefix, block_table, table_stride, seqlens, softmax_scale,
                             sinks, out, lse, workspace, workspace_bytes, stream_);
    }
    if (pl.prefix_partitions < 1 || pl.prefix_partitions > 4096 ||
        pl.prefix_groups != (static_cast<int64_t>(pl.B) * R + 127) / 128)
        return MLA_ERR_INVALID_ARG;
    const PrefixLayout lay = prefix_layout(pl);
    if (!workspace || workspace_bytes < lay.total || !aligned(workspace, 256)) return MLA_ERR_WORKSPACE;
    st = check_run_device(pl);
    if (st != MLA_OK) return st;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return MLA_ERR_CUDA;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    const uint64_t q_rows = static_cast<uint64_t>(pl.B) * R;

    // the prefix: one "sequence" per 128 rows of the batch, all reading the same
    // pages; every piece leaves a partial (a sink enters once, at the merge)
    mla_plan pre = pl;
    pre.kernel = MLA_KERNEL_PAIR;
    pre.B = pl.prefix_groups;
    pre.Sq = 1;
    pre.H = 128;
    pre.L_max = pl.prefix_max;
    pre.group_rows = 128;
    pre.num_groups = 1;
    pre.num_partitions = pl.prefix_partitions;
    mla::MainArgs ap;
    main_args(ap, pre, prefix_len, softmax_scale, nullptr, out, lse, workspace, lay.pre_lse, lay.pre_o);
    mla::PagedArgs pp = paged_args(pre, prefix_len, prefix_table, 0, num_pages, true);
    pp.len_stride = 0;
    pp.whole_slot = 2 * pl.prefix_partitions;
    pp.cut_tiles = kPartialCutTiles;
    st = launch_mla_paged(enc, pre, q, q_rows, kv_pages, ap, pp,
                          128ull * (2ull * pl.prefix_partitions + pl.prefix_groups), stream);
    if (st != MLA_OK) {
        cudaGetLastError();
        return st;
    }
    // the sequences' own keys, on the SMs that the prefix's launch leaves
    mla::MainArgs ao;
    main_args(ao, pl, seqlens, softmax_scale, nullptr, out, lse, workspace, lay.own_lse, lay.own_o);
    mla::PagedArgs po = paged_args(pl, seqlens, block_table, table_stride, num_pages, pl.kernel == MLA_KERNEL_PAIR);
    po.whole_slot = 2 * pl.num_partitions;
    po.cut_tiles = kPartialCutTiles;
    st = launch_mla_paged(enc, pl, q, q_rows, kv_pages, ao, po,
                          static_cast<uint64_t>(R) * (2ull * pl.num_partitions + pl.B), stream, true);
    if (st != MLA_OK) {
        cudaGetLastError();
        return st;
    }
    mla::PrefixCombineArgs c;
    c.B = pl.B;
    c.R = R;
    c.H = pl.H;
    c.P_own = pl.num_partitions;
    c.P_pre = pl.prefix_partitions;
    c.groups = pl.prefix_groups;
    c.out = ao.out;
    c.lse = lse;
    c.own_o = ao.part_o;
    c.own_lse = ao.part_lse;
    c.pre_o = ap.part_o;
    c.pre_lse = ap.part_lse;
    c.sinks = sinks;
    return launch_dependent(mla::mla_prefix_combine_kernel, combine_grid(pl), mla::kCombineThreads, stream, 0, c, po,
                            pp);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Appending to a paged cache.
// ---------------------------------------------------------------------------

namespace {

// Whether two of T x H rows of `width` elements, at t * token + h * head, share one.
bool rows_overlap(int64_t T, int64_t token, int64_t H, int64_t head, int64_t width) {
    token = token < 0 ? -token : token;
    head = head < 0 ? -head : head;
    if (T < 2) token = (H - 1) * head + width;
    if (H < 2) head = (T - 1) * token + width;
    if (head >= width && token >= (H - 1) * head + width) return false;
    if (token >= width && head >= (T - 1) * token + width) return false;
    // neither lies in the other's gaps as a block: the row nearest to h heads on, for every h
    if (token < width || head < width) return true;
    for (int64_t h = 1; h < H; ++h) {
        const int64_t t = std::min(h * head / token, T - 1), rest = h * head - t * token;
        if (rest < width || (t + 1 < T && token - rest < width)) return true;
    }
    return false;
}

// Checks what both kinds of append share and fills the kernel's arguments.
mla_status append_args(const mla_append* p, bool mha, mla::AppendArgs& a) {
    if (!p || !p->seqlens || !p->block_table || !p->cos_sin || !p->k_pages) return MLA_ERR_INVALID_ARG;
    if (p->T != 0 && (!p->k || !p->v || (p->H > 0 && (!p->q_in || !p->q_out)))) return MLA_ERR_INVALID_ARG;
    if (mha && !p->v_pages) return MLA_ERR_INVALID_ARG;
    if (p->B < 1 || p->T < 0 || p->page_size < 1 || p->num_pages < 1 || p->table_width < 1 || p->table_stride < 0 ||
        p->num_positions < 1 || p->H < 0 || p->H > 65535 || (p->interleaved != 0 && p->interleaved != 1))
        return MLA_ERR_INVALID_ARG;
    if (mha ? (p->Hkv < 1 || p->Hkv > 65535 || p->rope_dim < 16 || p->rope_dim > 128 || p->rope_dim % 16 != 0)
            : p->rope_dim != 64)
        return MLA_ERR_INVALID_ARG;
    if (!p->cu_tokens && p->T % p->B != 0) return MLA_ERR_INVALID_ARG;
    if (mha ? p->kv_scale != 0.f : !(std::isfinite(p->kv_scale) && p->kv_scale >= 0.f)) return MLA_ERR_INVALID_ARG;
    if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->k_pages, 16) || !aligned(p->v_pages, 16) ||
        !aligned(p->q_in, 16) || !aligned(p->q_out, 16) || !aligned(p->cos_sin, 16) || !aligned(p->seqlens, 4) ||
        !aligned(p->cu_tokens, 4) || !aligned(p->block_table, 4) || !aligned(p->status, 4))
        return MLA_ERR_ALIGNMENT;
    const int64_t strides[] = {p->k_token_stride, p->k_head_stride, p->v_token_stride, p->v_head_stride,
                               p->q_in_token_stride, p->q_in_head_stride, p->q_out_token_stride, p->q_out_head_stride};
    for (int64_t s : strides)
        if (s % 8 != 0) return MLA_ERR_ALIGNMENT;
    if (p->T > 0 && p->H > 0 &&
        rows_overlap(p->T, p->q_out_token_stride, p->H, p->q_out_head_stride, mha ? 128 : 64))
        return MLA_ERR_INVALID_ARG;
    std::memset(&a, 0, sizeof a);
    a.B = p->B;
    a.T = p->T;
    a.per_seq = p->T / p->B;
    a.cu = p->cu_tokens;
    a.seqlens = p->seqlens;
    a.table = p->block_table;
    a.table_stride = p->table_stride;
    a.table_width = p->table_width;
    a.num_pages = p->num_pages;
    a.page_size = p->page_size;
    a.cos_sin = p->cos_sin;
    a.num_positions = p->num_positions;
    a.rot = p->rope_dim;
    a.status = p->status;
    a.k = static_cast<const __nv_bfloat16*>(p->k);
    a.k_token = p->k_token_stride;
    a.k_head = p->k_head_stride;
    a.v = static_cast<const __nv_bfloat16*>(p->v);
    a.v_token = p->v_token_stride;
    a.v_head = p->v_head_stride;
    a.q_in = static_cast<const __nv_bfloat16*>(p->q_in);
    a.qi_token = p->q_in_token_stride;
    a.qi_head = p->q_in_head_stride;
    a.q_out = static_cast<__nv_bfloat16*>(p->q_out);
    a.qo_token = p->q_out_token_stride;
    a.qo_head = p->q_out_head_stride;
    a.H = p->H;
    a.Hkv = p->Hkv;
    a.k_pages = p->k_pages;
    a.v_pages = static_cast<__nv_bfloat16*>(p->v_pages);
    a.kv_scale = p->kv_scale;
    // (of bf16 values: at most 2^128, at least 2^-133)
    a.kv_inv = p->kv_scale > 0x1p-100f && p->kv_scale < 0x1p100f ? 1.f / p->kv_scale : 0.f;
    return MLA_OK;
}

// A token's tasks go to so many warps that there are about 8 an SM in all: 2178
// tokens of 6 tasks, kv in L2, take 10.6 us so (2 tasks a warp: 11.8, one: 13.2).
constexpr int64_t kAppendWarpsPerSm = 8;

mla_status launch_append(void (*kernel)(const mla::AppendArgs), const mla::AppendArgs& a, int tasks,
                         cudaStream_t stream) {
    if (a.T == 0) return MLA_OK;
    mla_plan any;
    any.device = -1;
    const mla_status st = check_run_device(any);
    if (st != MLA_OK) return st;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return MLA_ERR_CUDA;
    }
    const int64_t per = mla::kAppendThreads / 32;
    const int64_t parts = std::min<int64_t>(tasks, (kAppendWarpsPerSm * sms + a.T - 1) / a.T);
    const dim3 grid(static_cast<unsigned>((a.T + per - 1) / per), static_cast<unsigned>(parts));
    kernel<<<grid, mla::kAppendThreads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

mla_status mla_append_rows(const mla_append* args, const int32_t* prefix_len, void* stream) {
    mla::AppendArgs a;
    const mla_status st = append_args(args, false, a);
    if (st != MLA_OK) return st;
    if (!aligned(prefix_len, 4)) return MLA_ERR_ALIGNMENT;
    a.prefix_len = prefix_len;
    const int per = mla::HeadRows<64>::kHeads, tasks = 1 + (a.H + per - 1) / per;
    const bool fp8 = a.kv_scale > 0.f, il = args->interleaved != 0;
    return launch_append(fp8 ? (il ? mla::mla_cache_append_kernel<true, true> : mla::mla_cache_append_kernel<true, false>)
                             : (il ? mla::mla_cache_append_kernel<false, true> : mla::mla_cache_append_kernel<false, false>),
                         a, tasks, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

mla_status mla_cache_append(const mla_append* args, void* stream) { return mla_append_rows(args, nullptr, stream); }

mla_status mla_cache_append_prefix(const mla_append* args, const int32_t* prefix_len, void* stream) {
    if (!prefix_len) return MLA_ERR_INVALID_ARG;
    return mla_append_rows(args, prefix_len, stream);
}

mla_status mha_cache_append(const mla_append* args, void* stream) {
    mla::AppendArgs a;
    const mla_status st = append_args(args, true, a);
    if (st != MLA_OK) return st;
    const int per = mla::HeadRows<128>::kHeads, tasks = 2 * ((a.Hkv + per - 1) / per) + (a.H + per - 1) / per;
    return launch_append(args->interleaved ? mla::mha_cache_append_kernel<true> : mla::mha_cache_append_kernel<false>,
                         a, tasks, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
