"""GPU tests of the paged cache: decode over pages with a window and first tokens (bf16 and E4M3 latent pages, key and
value pages of grouped kv heads), decode of a batch with a shared prefix, and appending with the rotation, each against
a plain implementation in 64 bits on the same inputs, and of their refusals.

Tolerances.  Scores accumulate n products of the key's width in fp32, so each is off by at most
n 2^-24 scale sum |q k| =: delta (first order), and so is lse; its sum and its logarithm add a few 2^-23 of its value.
The weights a row multiplies its values with are rounded to bf16 (2^-8 relative; E4M3 pages: two E4M3 terms, 2^-4 of
2^-4, of a weight rounded to f16 at most, 2^-11, and 2^-14 of the largest weight where the second term has no more
bits), so with A = sum p |v| an output is off by at most (2^-8 + 2 delta) A, and by 2^-8 of itself from its own rounding.
2^-20 stands for the fp32 steps of the merges.  E4M3 pages: a query row, scaled so that its largest element is in
[224, 448], is carried as two or three E4M3 terms.  Two hold the 8 bits of a bf16 exactly unless its last bit is below
E4M3's smallest step 2^-9, and are off by half of that otherwise: 2^-10 / 224 of the row's largest element, in each of the
products.  Rows of a page that no token sees hold NaN (or the NaN code), and so do outputs before a call.
"""
import math

import pytest
import torch

from mla_decode_attention_11_b200 import binding as M

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"mla": 576, "mla_fp8": 576, "mha": 128}


class Pages:
    """A cache of pages in random order, NaN in every row, with rows of sequences written where they belong."""

    def __init__(self, kind, lengths, page, Hkv=1, seed=0, spare=2, width=None, table_pad=0):
        self.kind, self.page, self.lengths = kind, page, lengths
        g = torch.Generator(device=DEV).manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        self.num = sum(need) + spare
        order = torch.randperm(self.num, generator=g, device=DEV).to(torch.int32)
        width = max(1, max(need)) if width is None else width
        whole = torch.full((len(need), width + table_pad), -1, dtype=torch.int32, device=DEV)
        self.table = whole[:, :width]
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        shape = (self.num, page, 576) if kind != "mha" else (self.num, page, Hkv, 128)
        self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
        self.v = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV) if kind == "mha" else self.k
        self.scale = 1.0
        if kind == "mla_fp8":
            self.k = torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV)
            self.v, self.scale = self.k, 1.0 / 64
        self.gen = g

    def rows_of(self, table_row, n):
        j = torch.arange(n, device=DEV)
        return table_row.long()[j // self.page] * self.page + j % self.page

    def fill(self, table_row, n, only=None):
        """Random rows for positions 0..n-1 (`only`: a mask of the positions to write)."""
        at = self.rows_of(table_row, n)
        if only is not None:
            at = at[only]
        for x in {id(self.k): self.k, id(self.v): self.v}.values():
            r = torch.randn((at.numel(), *x.shape[2:]), generator=self.gen, device=DEV)
            if self.kind == "mla_fp8":
                r = (r * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            x.flatten(0, 1)[at] = r.to(x.dtype)

    def double(self, table_row, n):
        """(keys, values) [n, Hkv, D] in 64 bits."""
        at = self.rows_of(table_row, n)
        k, v = (x.flatten(0, 1)[at] for x in (self.k, self.v))
        if self.kind == "mla_fp8":
            k = v = k.view(torch.float8_e4m3fn).double() * self.scale
        k, v = k.double(), v.double()
        return (k, v) if self.kind == "mha" else (k[:, None], v[:, None, :512])


def seen_mask(L, Sq, window, first):
    j = torch.arange(L, device=DEV)[None]
    p = torch.arange(L - Sq, L, device=DEV)[:, None]
    m = j <= p
    if window:
        m = m & ((j > p - window) | (j < first))
    return m


def reference(q, seqs, masks, scale, sinks, values):
    """q [B, Sq, H, D] and per sequence (k, v) [n, Hkv, D] and its mask [Sq, n] -> out, lse, and their tolerances."""
    B, Sq, H, D = q.shape
    out = torch.zeros(B, Sq, H, values, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Sq, H), -math.inf, dtype=torch.float64, device=DEV)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for b, ((k, v), mask) in enumerate(zip(seqs, masks)):
        n, Hkv = k.shape[:2]
        gq = H // Hkv
        qq = q[b].double().view(Sq, Hkv, gq, D)
        seen = mask[:, None, None, :].expand(Sq, Hkv, gq, n)
        used = mask.any(0)
        k, v = torch.where(used[:, None, None], k, 0.0), torch.where(used[:, None, None], v, 0.0)
        s = torch.einsum("thgd,nhd->thgn", qq, k) * scale
        s = torch.where(seen, s, -math.inf)
        delta = torch.einsum("thgd,nhd->thgn", qq.abs(), k.abs()) * (abs(scale) * D * 2.0 ** -24)
        if reference.fp8:
            delta = delta + torch.einsum("thgd,nhd->thgn", qq.abs().amax(-1, keepdim=True).expand_as(qq), k.abs()) * (
                abs(scale) * 2.0 ** -10 / 224)
        delta = torch.where(seen, delta, 0.0).amax(-1) if n else torch.zeros(Sq, Hkv, gq, device=DEV).double()
        sk = None if sinks is None else sinks.double().view(1, Hkv, gq, 1).expand(Sq, Hkv, gq, 1)
        full = s if sk is None else torch.cat([s, sk], -1)
        if full.shape[-1] == 0:
            continue
        l = torch.logsumexp(full, -1)
        p = torch.where(l[..., None] == -math.inf, 0.0, torch.exp(s - torch.where(l == -math.inf, 0.0, l)[..., None]))
        o = torch.einsum("thgn,nhd->thgd", p, v)
        a = torch.einsum("thgn,nhd->thgd", p, v.abs())
        out[b], lse[b] = o.reshape(Sq, H, values), l.reshape(Sq, H)
        d = delta[..., None]
        # E4M3 weights: 2^-14 of the row's largest weight, at most p.max(), for each key
        small = p.amax(-1, keepdim=True) * torch.einsum("thgn,nhd->thgd", seen.double(), v.abs()) if n else a
        tol_o[b] = ((2.0 ** -8 + 2.0 ** -11 * reference.fp8 + 2 * d + 2.0 ** -20) * a + 2.0 ** -8 * o.abs() + 2.0 ** -14 * small * reference.fp8
                    ).reshape(Sq, H, values)
        tol_l[b] = torch.where(l == -math.inf, 0.0, delta + 2.0 ** -20 * (1 + l.abs())).reshape(Sq, H)
    return out, lse, tol_o, tol_l


reference.fp8 = 0.0


def close(out, lse, ref, what=""):
    ro, rl, to, tl = ref
    assert torch.isfinite(out.float()).all(), what
    worst = ((out.double() - ro).abs() - to).max().item()
    assert worst <= 0, f"{what}: out is {worst:.3e} past its tolerance"
    empty = rl == -math.inf
    assert torch.equal(lse == -math.inf, empty), what
    worst = ((lse.double() - rl).abs() - tl)[~empty]
    assert worst.numel() == 0 or worst.max().item() <= 0, f"{what}: lse is {worst.max().item():.3e} past its tolerance"


def blank(B, Sq, H, values):
    return (torch.full((B, Sq, H, values), float("nan"), dtype=torch.bfloat16, device=DEV),
            torch.full((B, Sq, H), float("nan"), dtype=torch.float32, device=DEV))


def make_window(kind, lengths, Sq, H, Hkv, page, window, first, sinks, seed, scale=None, L_max=None, parts=0,
                table_pad=0):
    B, D, values = len(lengths), DT[kind], 128 if kind == "mha" else 512
    L_max = L_max or max(1, max(lengths))
    pages = Pages(kind, lengths, page, Hkv, seed, width=-(-L_max // page), table_pad=table_pad)
    masks = [seen_mask(L, Sq, window, first) for L in lengths]
    for b, L in enumerate(lengths):
        if L:
            pages.fill(pages.table[b], L, masks[b].any(0))
    # pages without a visible key need no entry
    for b, L in enumerate(lengths):
        used = masks[b].any(0)
        for e in range(-(-L // page)):
            if not used[e * page:(e + 1) * page].any():
                pages.table[b, e] = -7
    seqs = []
    for b, L in enumerate(lengths):
        row = pages.table[b].clamp_min(0)
        seqs.append(pages.double(row, L))
    q = torch.randn(B, Sq, H, D, generator=pages.gen, device=DEV).bfloat16()
    sk = torch.randn(H, generator=pages.gen, device=DEV) * 2 if sinks else None
    if sinks:
        sk[0] = -math.inf
    scale = D ** -0.5 if scale is None else scale
    kw = dict(window=window, first_tokens=first, device=0, num_partitions=parts)
    if kind == "mha":
        plan = M.mha_decode_plan_paged(B, Sq, H, Hkv, L_max, page, **kw)
    else:
        plan = (M.mla_decode_plan_paged if kind == "mla" else M.mla_decode_plan_paged_fp8)(B, Sq, H, L_max, page, **kw)
    sl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    reference.fp8 = 1.0 if kind == "mla_fp8" else 0.0
    ref = reference(q, seqs, masks, scale, sk, values)
    ws = M.alloc_workspace(plan)

    def run(out, lse, stream=None):
        if kind == "mha":
            M.mha_decode_run_paged(plan, q, pages.k, pages.v, pages.table, sl, scale, out, lse, ws, sinks=sk,
                                   stream=stream)
        elif kind == "mla":
            M.mla_decode_run_paged(plan, q, pages.k, pages.table, sl, scale, out, lse, ws, sinks=sk, stream=stream)
        else:
            M.mla_decode_run_paged_fp8(plan, q, pages.k, pages.scale, pages.table, sl, scale, out, lse, ws, sinks=sk,
                                       stream=stream)
    return run, ref, blank(B, Sq, H, values), (plan, ws, pages, sl, q)


def check_window(*args, **kw):
    run, ref, (out, lse), (plan, ws, *_) = make_window(*args, **kw)
    run(out, lse)
    M.mla_decode_check(plan, ws)
    close(out, lse, ref, str(args))
    return out, lse


LENGTHS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 255, 256, 300, 700]


@pytest.mark.parametrize("parts", [0, 1, 7])
@pytest.mark.parametrize("window,first", [(0, 0), (1, 0), (1, 1), (40, 0), (40, 5), (128, 130), (200, 16), (5000, 3)])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("H", [16, 128])
def test_window_mla(cuda_device, H, page, window, first, parts):
    check_window("mla", LENGTHS, 1, H, 1, page, window, first, False, seed=page + window, parts=parts)


@pytest.mark.parametrize("window,first", [(0, 0), (1, 0), (3, 2), (100, 33)])
@pytest.mark.parametrize("page", [16, 32, 192])
@pytest.mark.parametrize("Sq,H", [(2, 16), (3, 16), (2, 32), (16, 16), (2, 128), (3, 64), (5, 128)])
def test_window_mla_tokens(cuda_device, Sq, H, page, window, first):
    """Several query tokens, among them tokens before the sequence's first key (which see nothing)."""
    check_window("mla", LENGTHS, Sq, H, 1, page, window, first, True, seed=Sq + H + page, parts=5)


@pytest.mark.parametrize("parts", [0, 1, 7])
@pytest.mark.parametrize("window,first", [(0, 0), (1, 1), (40, 5), (200, 16)])
@pytest.mark.parametrize("page", [16, 96, 128])
@pytest.mark.parametrize("Sq,H", [(1, 16), (2, 16), (3, 32), (1, 128), (2, 64), (3, 128)])
def test_window_mla_fp8(cuda_device, Sq, H, page, window, first, parts):
    check_window("mla_fp8", LENGTHS, Sq, H, 1, page, window, first, Sq > 1, seed=page + window, parts=parts)


@pytest.mark.parametrize("window,first", [(0, 0), (1, 1), (40, 5), (200, 16)])
@pytest.mark.parametrize("page", [16, 64, 384])
@pytest.mark.parametrize("Sq,H,Hkv", [(1, 32, 8), (1, 8, 8), (1, 7, 7), (2, 16, 2), (4, 24, 3), (1, 32, 1), (3, 1, 1)])
def test_window_mha(cuda_device, Sq, H, Hkv, page, window, first):
    for parts in (0, 6):
        check_window("mha", LENGTHS, Sq, H, Hkv, page, window, first, Sq == 1, seed=H + page, parts=parts)


@pytest.mark.parametrize("kind,H,Hkv", [("mla", 16, 1), ("mla", 128, 1), ("mla_fp8", 16, 1), ("mla_fp8", 128, 1), ("mha", 32, 8)])
def test_long_window(cuda_device, kind, H, Hkv):
    """Lengths far past the window, a strided block table, a scale other than the usual one, negative and zero."""
    lengths = [30000, 12345, 4096, 4097, 9000, 1]
    for scale in (0.03, -0.02, 0.0):
        check_window(kind, lengths, 1, H, Hkv, 64, 4096, 4, False, seed=1, scale=scale, table_pad=3)
    check_window(kind, lengths, 2, H, Hkv, 64, 511, 129, True, seed=2)


def test_many_short_sequences(cuda_device):
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 200, (700,), generator=g).tolist()
    for kind, H, Hkv in (("mla", 16, 1), ("mla", 128, 1), ("mla_fp8", 16, 1), ("mla_fp8", 128, 1), ("mha", 8, 2)):
        check_window(kind, lengths, 1, H, Hkv, 32, 50, 3, False, seed=4)


def test_large_cache_offsets(cuda_device):
    """Pages past 2^31 elements of the cache."""
    page, pages = 256, 15000
    kv = torch.zeros(pages, page, 576, dtype=torch.bfloat16, device=DEV)
    L = 1000
    table = torch.tensor([[pages - 1, 3, pages - 2, 14999 - 7]], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    for e in range(4):
        kv[int(table[0, e])] = torch.randn(page, 576, generator=g, device=DEV).bfloat16()
    k = kv[table[0].long()].flatten(0, 1)[:L].double()
    for H in (16, 128):
        q = torch.randn(1, 1, H, 576, generator=g, device=DEV).bfloat16()
        plan = M.mla_decode_plan_paged(1, 1, H, L, page, device=0)
        ws = M.alloc_workspace(plan)
        out, lse = blank(1, 1, H, 512)
        sl = torch.tensor([L], dtype=torch.int32, device=DEV)
        M.mla_decode_run_paged(plan, q, kv, table, sl, 576 ** -0.5, out, lse, ws)
        M.mla_decode_check(plan, ws)
        reference.fp8 = 0.0
        close(out, lse, reference(q, [(k[:, None], k[:, None, :512])], [seen_mask(L, 1, 0, 0)], 576 ** -0.5, None, 512))


@pytest.mark.parametrize("kind,H,Hkv", [("mla", 16, 1), ("mla", 128, 1), ("mla_fp8", 16, 1), ("mla_fp8", 128, 1), ("mha", 32, 8)])
def test_same_result_again_on_a_stream_and_in_a_graph(cuda_device, kind, H, Hkv):
    run, ref, (out, lse), (plan, ws, *_) = make_window(kind, [5, 900, 0, 333, 2000], 1, H, Hkv, 16, 300, 4, True, seed=9)
    run(out, lse)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    out2, lse2 = blank(*out.shape[:3], out.shape[3])
    with torch.cuda.stream(side):
        run(out2, lse2)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    out3, lse3 = blank(*out.shape[:3], out.shape[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out3, lse3)
    for _ in range(3):
        out3.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    M.mla_decode_check(plan, ws)
    assert torch.equal(out, out3) and torch.equal(lse, lse3)
    close(out, lse, ref)


def test_bad_pages_and_lengths_are_flagged(cuda_device):
    """An entry outside the cache reads as zeros and is reported; a length past L_max is clamped and reported."""
    for kind, H, Hkv in (("mla", 16, 1), ("mla", 128, 1), ("mla_fp8", 32, 1), ("mla_fp8", 128, 1), ("mha", 8, 2)):
        run, ref, (out, lse), (plan, ws, pages, sl, q) = make_window(kind, [100, 300, 260], 1, H, Hkv, 64, 0, 0, False, 11)
        for bad in (-1, pages.num, 2 ** 31 - 1, -2 ** 31):
            good = int(pages.table[1, 2])
            pages.table[1, 2] = bad
            run(out, lse)
            with pytest.raises(M.MlaError) as e:
                M.mla_decode_check(plan, ws)
            assert e.value.code == 8
            pages.table[1, 2] = good
            for b in (0, 2):  # the others are as they should be
                close(out[b:b + 1], lse[b:b + 1], [r[b:b + 1] for r in ref])
        sl[0] = plan.L_max + 1
        run(out, lse)
        with pytest.raises(M.MlaError) as e:
            M.mla_decode_check(plan, ws)
        assert e.value.code in (7, 8)  # the clamped length may also need pages that the table does not have
        sl[0] = 100
        run(out, lse)
        M.mla_decode_check(plan, ws)
        close(out, lse, ref)


@pytest.mark.parametrize("kind,H,Hkv", [("mla", 16, 1), ("mla", 128, 1), ("mla_fp8", 16, 1), ("mla_fp8", 128, 1), ("mha", 8, 2)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 300, 299])
def test_windows_around_the_longest_length(cuda_device, kind, H, Hkv, window):
    check_window(kind, [300, 299, 1, 0, 128], 2, H, Hkv, 32, window, 3, False, 13)


# unit 2 is the last that CTA 0 loads of a single tile of grouped kv heads (0: queries, 1: keys, 2: values)
@pytest.mark.parametrize("unit,parts", [(2, 0), (30, 1)])
@pytest.mark.parametrize("kind,H,Hkv", [("mla", 16, 1), ("mla", 128, 1), ("mla_fp8", 16, 1), ("mla_fp8", 128, 1), ("mha", 8, 2)])
def test_bounded_wait_timeout_reports_and_recovers(cuda_device, kind, H, Hkv, unit, parts):
    """The producer of CTA 0 arms a barrier and leaves out its load: the consumers' waits run out after 20 ms, every
    role unwinds, the run reports MLA_ERR_TIMEOUT and the next one on the same workspace is clean."""
    run, ref, (out, lse), (plan, ws, *_) = make_window(kind, [1000, 990], 1, H, Hkv, 64, 0, 0, False, 17, parts=parts)
    try:
        M.mla_decode_set_debug(wait_timeout_ns=20_000_000, stall_unit=unit)
        run(out, lse)
        with pytest.raises(M.MlaError) as e:
            M.mla_decode_check(plan, ws)
        assert e.value.code == 5
    finally:
        M.mla_decode_set_debug(0, -1)
    run(out, lse)
    M.mla_decode_check(plan, ws)
    close(out, lse, ref)


# ---------------------------------------------------------------- shared prefix

def make_prefix(lengths, Sq, H, P, page, sinks, seed, parts=0, prefix_max=None, L_max=None):
    B = len(lengths)
    L_max, prefix_max = L_max or max(1, max(lengths)), prefix_max or max(1, P)
    pages = Pages("mla", [*lengths, P], page, seed=seed, width=max(-(-L_max // page), -(-prefix_max // page)))
    prefix_table = pages.table[B].contiguous()
    masks = [seen_mask(L, Sq, 0, 0) for L in lengths]
    for b, L in enumerate(lengths):
        if L:
            pages.fill(pages.table[b], L, masks[b].any(0))
    if P:
        pages.fill(prefix_table, P)
    pk, pv = pages.double(prefix_table.clamp_min(0), P)
    seqs, seen = [], []
    for b, L in enumerate(lengths):
        k, v = pages.double(pages.table[b].clamp_min(0), L)
        seqs.append((torch.cat([pk, k]), torch.cat([pv, v])))
        seen.append(torch.cat([torch.ones(Sq, P, dtype=torch.bool, device=DEV), masks[b]], 1))
    q = torch.randn(B, Sq, H, 576, generator=pages.gen, device=DEV).bfloat16()
    sk = torch.randn(H, generator=pages.gen, device=DEV) * 2 if sinks else None
    scale = 576 ** -0.5
    reference.fp8 = 0.0
    ref = reference(q, seqs, seen, scale, sk, 512)
    plan = M.mla_decode_plan_prefix(B, Sq, H, L_max, prefix_max, page, device=0, num_partitions=parts)
    ws = M.alloc_workspace(plan)
    sl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    pl = torch.tensor([P], dtype=torch.int32, device=DEV)

    def run(out, lse):
        M.mla_decode_run_prefix(plan, q, pages.k, prefix_table, pl, pages.table[:B], sl, scale, out, lse, ws, sinks=sk)
    run.q = q
    return run, ref, blank(B, Sq, H, 512), (plan, ws, pages, sl, pl)


# a prefix planned as long as this has a launch of its own where a sequence has fewer than 128 query rows
LONG = 1 << 18


@pytest.mark.parametrize("parts", [0, 1, 7])
@pytest.mark.parametrize("P", [0, 1, 100, 128, 500, 2049])
@pytest.mark.parametrize("Sq,H,most", [(1, 16, 0), (1, 16, LONG), (3, 16, 0), (3, 16, LONG), (1, 64, LONG), (2, 32, 0),
                                       (1, 128, 0), (2, 128, 0)])
def test_prefix(cuda_device, Sq, H, most, P, parts):
    lengths = [0, 1, 2, 17, 128, 129, 400]
    run, ref, (out, lse), (plan, ws, *_) = make_prefix(lengths, Sq, H, P, 16 if P < 200 else 64, H == 16, seed=P + H,
                                                       parts=parts, prefix_max=most)
    assert (plan.prefix_partitions > 0) == (most == LONG)
    run(out, lse)
    M.mla_decode_check(plan, ws)
    close(out, lse, ref, f"{Sq} {H} {P} {parts}")


@pytest.mark.parametrize("most", [0, LONG])
@pytest.mark.parametrize("B,Sq,H", [(1, 1, 16), (9, 1, 16), (300, 1, 16), (64, 1, 128), (33, 2, 32)])
def test_prefix_batches(cuda_device, B, Sq, H, most):
    """Row groups of 128 that are not full, and more groups than partitions."""
    g = torch.Generator().manual_seed(B)
    lengths = torch.randint(0, 300, (B,), generator=g).tolist()
    run, ref, (out, lse), (plan, ws, *_) = make_prefix(lengths, Sq, H, 900, 64, True, seed=B, prefix_max=most)
    run(out, lse)
    M.mla_decode_check(plan, ws)
    close(out, lse, ref)


@pytest.mark.parametrize("most", [5000, LONG])
def test_prefix_shorter_than_planned_and_in_a_graph(cuda_device, most):
    """The prefix's length is read on the device: a captured call follows it."""
    run, ref, (out, lse), (plan, ws, pages, sl, pl) = make_prefix([30, 0, 200], 1, 64, 700, 32, False, seed=5,
                                                                  prefix_max=most, L_max=900)
    run(out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, lse)
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    M.mla_decode_check(plan, ws)
    close(out, lse, ref)
    pl.fill_(0)
    graph.replay()
    M.mla_decode_check(plan, ws)
    assert torch.count_nonzero(out[1]) == 0 and (lse[1] == -math.inf).all()
    pl.fill_(most + 1)
    graph.replay()
    with pytest.raises(M.MlaError) as e:
        M.mla_decode_check(plan, ws)
    assert e.value.code in (7, 8)


# ---------------------------------------------------------------- appending

def turned(x, table, pos, interleaved):
    """x [T, heads, W] in 64 bits, its first columns turned by the angles of pos [T]."""
    x = x.double().clone()
    cs = table[pos].double()[:, None]
    n = cs.shape[-1] // 2
    c, s = cs[..., :n], cs[..., n:]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    u, w = a * c - b * s, b * c + a * s
    if interleaved:
        x[..., 0:2 * n:2], x[..., 1:2 * n:2] = u, w
    else:
        x[..., :n], x[..., n:2 * n] = u, w
    return x


def turn_tolerance(x, n):
    """fp32 products and sum (3 2^-24 of |x0| + |x1| <= 2 max) and the rounding to bf16 (2^-8 of the result)."""
    big = x.double().abs().amax(-1, keepdim=True) * 2
    return lambda r: 2.0 ** -8 * r.abs() + 3 * 2.0 ** -24 * big


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


TOKENS = [([5], [5]), ([1, 1, 1], [1, 300, 40]), ([0, 3, 0, 17, 1], [0, 3, 9, 500, 1]), ([130, 0, 64], [130, 0, 64])]


def places(new, lengths, table, page):
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(new, lengths)]).to(DEV)
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).to(DEV)
    return pos, table.long()[seq, pos // page] * page + pos % page


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("H", [0, 1, 16, 33, 128])
def test_append_mla(cuda_device, H, page, fp8, interleaved):
    cos_sin = M.rope_table(600, 64, device=DEV)
    for case, (new, lengths) in enumerate(TOKENS):
        g = torch.Generator(device=DEV).manual_seed(case + H)
        pages = Pages("mla", lengths, page, seed=case)
        T = sum(new)
        row = rand(g, T, 600)  # the rows' parts are slices of a wider product
        latent, k_rope = row[:, 8:520], row[:, 520:584]
        q_rope = rand(g, T, H, 192)[..., 128:] if H else None
        q = rand(g, T, H, 576) if H else None
        q0 = None if q is None else q.clone()
        scale = 1 / 50 if fp8 else None
        kv = pages.k
        if fp8:
            kv = torch.randint(0, 256, pages.k.shape, generator=g, device=DEV).to(torch.uint8).view(torch.float8_e4m3fn)
        before = kv.view(torch.uint8).clone()
        cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
        sl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        plan = M.mla_decode_plan_paged(len(new), 1, 16, max(1, max(lengths)), 16, device=0)
        ws = M.alloc_workspace(plan)
        M.mla_cache_append(latent, k_rope, cos_sin, kv, pages.table, sl, cu_tokens=cu, q_rope=q_rope, q=q,
                           kv_scale=scale, interleaved=interleaved, workspace=ws)
        M.mla_decode_check(plan, ws)
        pos, at = places(new, lengths, pages.table, page)
        got = kv.flatten(0, 1)[at].double() if not fp8 else kv.view(torch.uint8).flatten(0, 1)[at].view(
            torch.float8_e4m3fn).double()
        rope = turned(k_rope[:, None], cos_sin, pos, interleaved)[:, 0]
        want = torch.cat([latent.double(), rope], 1)
        if fp8:
            # round to nearest of x / scale: 2^-4 of the value, half the smallest subnormal, and fp32 steps
            want = (want / float(torch.tensor(scale))).clamp(-448, 448)
            assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 + 1e-4).all()
            codes = (latent.float() / torch.tensor(scale, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(kv.view(torch.uint8).flatten(0, 1)[at][:, :512], codes)
        else:
            assert torch.equal(got[:, :512], latent.double())
            assert ((got[:, 512:] - rope).abs() <= turn_tolerance(k_rope, 64)(rope)).all()
        # everything else is as it was
        rest = torch.ones(kv.shape[0] * page, dtype=torch.bool, device=DEV)
        rest[at] = False
        assert torch.equal(kv.view(torch.uint8).flatten(0, 1)[rest], before.flatten(0, 1)[rest])
        if H:
            want = turned(q_rope, cos_sin, pos, interleaved)
            assert ((q[..., 512:].double() - want).abs() <= turn_tolerance(q_rope, 64)(want)).all()
            assert torch.equal(q[..., :512], q0[..., :512])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("H,Hkv,page", [(8, 8, 16), (32, 8, 64), (9, 1, 5), (0, 3, 16), (70, 35, 16)])
def test_append_mha(cuda_device, H, Hkv, page, rot, interleaved):
    cos_sin = M.rope_table(600, rot, device=DEV)
    for case, (new, lengths) in enumerate(TOKENS):
        g = torch.Generator(device=DEV).manual_seed(case + H)
        pages = Pages("mha", lengths, page, Hkv, seed=case)
        T = sum(new)
        # keys and values are slices of one projection's rows
        qkv = rand(g, T, H + 2 * Hkv, 128)
        q_in, k, v = qkv[:, :H] if H else None, qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        inplace = case % 2 == 1
        keep = qkv.clone()
        q_out = None if not H else q_in if inplace else torch.empty(T, H, 128, dtype=torch.bfloat16, device=DEV)
        cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
        sl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        M.mha_cache_append(k, v, cos_sin, pages.k, pages.v, pages.table, sl, cu_tokens=cu, q_in=q_in, q_out=q_out,
                           interleaved=interleaved)
        pos, at = places(new, lengths, pages.table, page)
        want = turned(keep[:, H:H + Hkv], cos_sin, pos, interleaved)
        got = pages.k.flatten(0, 1)[at].double()
        assert ((got - want).abs() <= turn_tolerance(keep[:, H:H + Hkv], rot)(want)).all()
        assert torch.equal(got[..., rot:], keep[:, H:H + Hkv, rot:].double())
        assert torch.equal(pages.v.flatten(0, 1)[at], keep[:, H + Hkv:])
        rest = torch.ones(pages.num * page, dtype=torch.bool, device=DEV)
        rest[at] = False
        assert torch.isnan(pages.k.flatten(0, 1)[rest].float()).all()
        assert torch.isnan(pages.v.flatten(0, 1)[rest].float()).all()
        if H:
            want = turned(keep[:, :H], cos_sin, pos, interleaved)
            assert ((q_out.double() - want).abs() <= turn_tolerance(keep[:, :H], rot)(want)).all()


@pytest.mark.parametrize("scale", [1 / 60, 1.0, 3.0, 0.0123, 2.0 ** -110, 2.0 ** 110, 1e-30, 7e29])
def test_append_quantises_every_value(cuda_device, scale):
    """Every finite bf16 value of the latent columns, and infinities and NaN, against a division in 32 bits."""
    bits = torch.arange(65536, device=DEV).to(torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).view(128, 512)
    kv = torch.zeros(8, 16, 576, dtype=torch.uint8, device=DEV)
    rope = torch.zeros(128, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    sl = torch.tensor([128], dtype=torch.int32, device=DEV)
    M.mla_cache_append(x, rope, M.rope_table(128, 64, device=DEV), kv, table, sl, kv_scale=scale)
    got = kv.flatten(0, 1)[:, :512].contiguous().view(torch.float8_e4m3fn).float()
    want = (x.float() / torch.tensor(scale, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    nan = torch.isnan(x.float())
    assert torch.isnan(got[nan]).all()
    assert torch.equal(got[~nan], want[~nan])


def test_append_uniform_padded_and_unplaced_tokens(cuda_device):
    """cu_tokens None: the same number for each; tokens past the last bound are padding; a token without a position or
    page is reported, and the others are written."""
    cos_sin = M.rope_table(100, 64, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    pages = Pages("mla", [64, 64, 64], 16)
    plan = M.mla_decode_plan_paged(3, 1, 16, 64, 16, device=0)
    ws = M.alloc_workspace(plan)
    row, q_rope = rand(g, 12, 576), rand(g, 12, 16, 64)
    q = torch.zeros(12, 16, 576, dtype=torch.bfloat16, device=DEV)
    sl = torch.tensor([4, 20, 64], dtype=torch.int32, device=DEV)
    M.mla_cache_append(row[:, :512], row[:, 512:], cos_sin, pages.k, pages.table, sl, q_rope=q_rope, q=q, workspace=ws)
    M.mla_decode_check(plan, ws)
    pos, at = places([4, 4, 4], [4, 20, 64], pages.table, 16)
    assert torch.equal(pages.k.flatten(0, 1)[at][:, :512], row[:, :512])
    # padding: 5 tokens, 3 + 1 of them of sequences
    pages = Pages("mla", [64, 64, 64], 16)
    cu = torch.tensor([0, 3, 3, 4], dtype=torch.int32, device=DEV)
    q.zero_()
    M.mla_cache_append(row[:5, :512], row[:5, 512:], cos_sin, pages.k, pages.table, sl, cu_tokens=cu, q_rope=q_rope[:5],
                       q=q[:5], workspace=ws)
    M.mla_decode_check(plan, ws)
    assert torch.count_nonzero(q[4:]) == 0 and torch.count_nonzero(q[3, :, 512:]) > 0
    assert int((~torch.isnan(pages.k.flatten(0, 1)[:, 0].float())).sum()) == 4
    # positions past the rotation table, below zero; pages past the table, outside the cache
    sl = torch.tensor([2, 101, 63], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 3, 5, 6], dtype=torch.int32, device=DEV)
    M.mla_cache_append(row[:6, :512], row[:6, 512:], cos_sin, pages.k, pages.table, sl, cu_tokens=cu, workspace=ws)
    with pytest.raises(M.MlaError) as e:
        M.mla_decode_check(plan, ws)
    assert e.value.code == 7
    assert torch.equal(pages.k.flatten(0, 1)[pages.table[0, 0] * 16][:512], row[1, :512])  # token 1 is at position 0
    for entry in (-1, pages.num, -2 ** 31):
        pages.table[2, 3] = entry
        q.zero_()
        M.mla_cache_append(row[:6, :512], row[:6, 512:], cos_sin, pages.k, pages.table,
                           torch.tensor([3, 5, 63], dtype=torch.int32, device=DEV), cu_tokens=cu, q_rope=q_rope[:6],
                           q=q[:6], workspace=ws)
        with pytest.raises(M.MlaError) as e:
            M.mla_decode_check(plan, ws)
        assert e.value.code == 8
        assert torch.count_nonzero(q[5, :, 512:]) > 0  # its queries are rotated all the same


def test_append_many_sequences_and_no_tokens(cuda_device):
    """Where a token's sequence is found among many, most of them without tokens."""
    g = torch.Generator().manual_seed(1)
    new = torch.randint(0, 3, (3000,), generator=g) * (torch.rand(3000, generator=g) < 0.3)
    lengths = (new + torch.randint(0, 20, (3000,), generator=g)).tolist()
    new = new.tolist()
    pages = Pages("mha", lengths, 16, 1)
    gd = torch.Generator(device=DEV).manual_seed(1)
    T = sum(new)
    k, v = rand(gd, T, 1, 128), rand(gd, T, 1, 128)
    cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    sl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    cos_sin = M.rope_table(64, 128, device=DEV)
    M.mha_cache_append(k, v, cos_sin, pages.k, pages.v, pages.table, sl, cu_tokens=cu)
    _, at = places(new, lengths, pages.table, 16)
    assert torch.equal(pages.v.flatten(0, 1)[at], v)
    assert int((~torch.isnan(pages.v.flatten(0, 1)[:, 0, 0].float())).sum()) == T
    before = pages.k.clone()
    M.mha_cache_append(k[:0], v[:0], cos_sin, pages.k, pages.v, pages.table, sl, cu_tokens=torch.zeros_like(cu))
    assert torch.equal(torch.nan_to_num(before), torch.nan_to_num(pages.k))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fp8,H,page", [(False, 16, 16), (False, 128, 16), (True, 16, 16), (True, 128, 32)])
def test_append_then_decode(cuda_device, fp8, H, page):
    """Three steps of a server: prompts of odd lengths are appended, then tokens one by one, and each step's decode
    equals the 64-bit one over all that was appended; the whole step is captured once and replayed."""
    g = torch.Generator(device=DEV).manual_seed(2)
    prompts, window, first = [37, 1, 200, 90], 64, 4
    B, total = 4, [n + 3 for n in prompts]
    pages = Pages("mla_fp8" if fp8 else "mla", total, page, seed=3)
    cos_sin = M.rope_table(400, 64, device=DEV)
    scale, kv_scale = 576 ** -0.5, pages.scale if fp8 else None
    row = rand(g, sum(prompts), 576)
    cu = torch.tensor([0] + torch.tensor(prompts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    sl = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    M.mla_cache_append(row[:, :512], row[:, 512:], cos_sin, pages.k, pages.table, sl, cu_tokens=cu, kv_scale=kv_scale)
    make = M.mla_decode_plan_paged_fp8 if fp8 else M.mla_decode_plan_paged
    plan = make(B, 1, H, max(total), page, window=window, first_tokens=first, device=0)
    ws = M.alloc_workspace(plan)
    out, lse = blank(B, 1, H, 512)
    new, q_rope, q = rand(g, B, 576), rand(g, B, H, 64), rand(g, B, H, 576)

    def step():
        sl.add_(1)
        M.mla_cache_append(new[:, :512], new[:, 512:], cos_sin, pages.k, pages.table, sl, q_rope=q_rope, q=q,
                           kv_scale=kv_scale, workspace=ws)
        if fp8:
            M.mla_decode_run_paged_fp8(plan, q[:, None], pages.k, kv_scale, pages.table, sl, scale, out, lse, ws)
        else:
            M.mla_decode_run_paged(plan, q[:, None], pages.k, pages.table, sl, scale, out, lse, ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        if i:
            new.copy_(rand(g, B, 576)), q_rope.copy_(rand(g, B, H, 64))
            graph.replay()
        M.mla_decode_check(plan, ws)
        lengths = [n + 1 + i for n in prompts]
        assert sl.tolist() == lengths
        want = turned(q_rope, cos_sin, sl.long() - 1, True)
        assert ((q[..., 512:].double() - want).abs() <= turn_tolerance(q_rope, 64)(want)).all()
        reference.fp8 = 1.0 if fp8 else 0.0
        seqs = [pages.double(pages.table[b], L) for b, L in enumerate(lengths)]
        close(out, lse, reference(q[:, None], seqs, [seen_mask(L, 1, window, first) for L in lengths], scale, None, 512),
              f"step {i}")


@pytest.mark.parametrize("most", [0, LONG])
@pytest.mark.parametrize("H", [16, 128])
def test_prefix_equals_whole_sequences(cuda_device, H, most):
    """The shared-prefix decode of a batch against the plain paged decode of the same sequences with the prefix's pages
    in front of their own: both are within their tolerances of the same values, so within twice them of each other."""
    P, page, lengths = 256, 64, [1, 100, 64]
    run, ref, (out, lse), (plan, ws, pages, sl, pl) = make_prefix(lengths, 1, H, P, page, False, seed=8, prefix_max=most)
    run(out, lse)
    M.mla_decode_check(plan, ws)
    close(out, lse, ref)
    table = torch.cat([pages.table[3, :P // page].expand(3, -1), pages.table[:3, :2]], 1).contiguous()
    whole = M.mla_decode_plan_paged(3, 1, H, P + 128, page, device=0)
    ws = M.alloc_workspace(whole)
    out2, lse2 = blank(3, 1, H, 512)
    M.mla_decode_run_paged(whole, run.q, pages.k, table, sl + P, 576 ** -0.5, out2, lse2, ws)
    M.mla_decode_check(whole, ws)
    close(out2, lse2, ref)


def test_calls_on_two_streams_at_once(cuda_device):
    """Two-launch prefix decodes on one stream while paged decodes of every kernel run on another, each with a workspace
    of its own: the same bits as one after the other."""
    jobs = [make_prefix([40, 0, 300, 128] * 10, 1, 16, 900, 64, True, seed=1, prefix_max=LONG),
            make_prefix([40, 0, 300] * 5, 1, 128, 500, 64, False, seed=2)]
    jobs += [make_window(kind, [700, 5, 2000, 90], 1, H, Hkv, 64, 256, 4, False, 3)
             for kind, H, Hkv in (("mla", 16, 1), ("mla", 128, 1), ("mla_fp8", 32, 1), ("mla_fp8", 128, 1), ("mha", 8, 2))]
    alone = []
    for run, ref, (out, lse), (plan, ws, *_) in jobs:
        run(out, lse)
        M.mla_decode_check(plan, ws)
        alone.append((out.clone(), lse.clone()))
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (run, ref, (out, lse), _) in enumerate(jobs):
            with torch.cuda.stream(streams[0 if i < 2 else 1]):
                run(out, lse)
    torch.cuda.synchronize()
    for (run, ref, (out, lse), (plan, ws, *_)), (o, l) in zip(jobs, alone):
        M.mla_decode_check(plan, ws)
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_refusals(cuda_device):
    pages = Pages("mla", [64, 64], 16)
    plan = M.mla_decode_plan_paged(2, 1, 16, 64, 16, device=0)
    ws, sl = M.alloc_workspace(plan), torch.tensor([64, 64], dtype=torch.int32, device=DEV)
    q = torch.zeros(2, 1, 16, 576, dtype=torch.bfloat16, device=DEV)
    out, lse = blank(2, 1, 16, 512)

    def run(plan=plan, q=q, kv=pages.k, table=pages.table, sl=sl, out=out, lse=lse, ws=ws, sinks=None):
        M.mla_decode_run_paged(plan, q, kv, table, sl, 0.04, out, lse, ws, sinks=sinks)
    pages.k.zero_()
    run()
    M.mla_decode_check(plan, ws)
    with pytest.raises(ValueError):
        run(q=q.cpu())
    with pytest.raises(TypeError):
        run(q=q.half())
    with pytest.raises(ValueError):
        run(kv=pages.k[:, :8])
    with pytest.raises(TypeError):
        run(table=pages.table.long())
    with pytest.raises(ValueError):
        run(table=pages.table.t().contiguous().t())
    with pytest.raises(ValueError):
        run(sl=sl[:1])
    with pytest.raises(ValueError):
        run(out=out[..., :256])
    with pytest.raises(ValueError):
        run(sinks=torch.zeros(15, device=DEV))
    with pytest.raises(M.MlaError) as e:
        run(table=pages.table[:, :3])  # too narrow for L_max
    assert e.value.code == 1
    with pytest.raises(M.MlaError) as e:
        run(ws=ws[:1024])
    assert e.value.code == 6
    with pytest.raises(M.MlaError) as e:
        run(plan=M.mla_decode_plan_paged_fp8(2, 1, 16, 64, 16, device=0))
    assert e.value.code == 1
    with pytest.raises(M.MlaError) as e:
        run(kv=pages.k[:0])  # no pages
    assert e.value.code == 1

    cos_sin = M.rope_table(64, 64, device=DEV)
    row, qr = torch.zeros(2, 576, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    qq = torch.zeros(2, 4, 576, dtype=torch.bfloat16, device=DEV)
    ok = dict(latent=row[:, :512], k_rope=row[:, 512:], cos_sin=cos_sin, kv_pages=pages.k, block_table=pages.table,
              seqlens=sl, q_rope=qr, q=qq)
    M.mla_cache_append(**ok)
    for bad, error in ((dict(latent=row[:, 1:513]), M.MlaError),          # rows not 16-byte aligned
                       (dict(latent=row[:, :512].float()), TypeError), (dict(k_rope=row[:1, 512:]), ValueError),
                       (dict(cos_sin=cos_sin[:, :32].contiguous()), ValueError), (dict(kv_scale=0.1), ValueError),
                       (dict(kv_pages=pages.k.view(torch.uint8)[..., :576].contiguous()), ValueError),
                       (dict(q=None), ValueError), (dict(q_rope=None), ValueError),
                       (dict(q=qq[:, :1].expand(2, 4, 576)), ValueError),
                       (dict(q_rope=qr.cpu()), ValueError), (dict(seqlens=sl[:1]), ValueError),
                       (dict(cu_tokens=sl), ValueError), (dict(cos_sin=cos_sin.cpu()), ValueError)):
        with pytest.raises(error):
            M.mla_cache_append(**{**ok, **bad})
    with pytest.raises(M.MlaError):  # 3 tokens of 2 sequences without cu_tokens
        three = torch.zeros(3, 576, dtype=torch.bfloat16, device=DEV)
        M.mla_cache_append(three[:, :512], three[:, 512:], cos_sin, pages.k, pages.table, sl)
    heads = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device=DEV)
    kp = torch.zeros(4, 16, 4, 128, dtype=torch.bfloat16, device=DEV)
    for n in (8, 24, 136):
        with pytest.raises(M.MlaError):
            M.mha_cache_append(heads, heads, torch.zeros(64, n, device=DEV), kp, kp.clone(), pages.table, sl)


def test_append_refuses_scales_and_workspaces(cuda_device):
    """An E4M3 cache's scale that fp32 cannot hold is refused (rounded to 0 it would stand for a cache of bf16 rows,
    twice as long), and a workspace without room for the status words."""
    table, sl = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([1], dtype=torch.int32, device=DEV)
    row = torch.ones(1, 576, dtype=torch.bfloat16, device=DEV)
    codes = torch.full((2, 16, 576), 0x55, dtype=torch.uint8, device=DEV)
    call = lambda **kw: M.mla_cache_append(row[:, :512], row[:, 512:], M.rope_table(16, 64, device=DEV),
                                           codes, table, sl, **kw)
    for bad in (0.0, -1.0, math.nan, math.inf, 1e-60, 1e-46, 1e60, None):
        with pytest.raises(ValueError):
            call(kv_scale=bad)
    for words in (0, 63):
        with pytest.raises(ValueError):
            call(kv_scale=1.0, workspace=torch.zeros(words, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert bool((codes == 0x55).all())
    call(kv_scale=2.0 ** -149)
    assert bool((codes[0, 0] == 0x7E).sum() >= 512) and bool((codes[0, 1:] == 0x55).all()) and bool((codes[1] == 0x55).all())


@pytest.mark.parametrize("kind", ["mla", "mla_fp8", "mha"])
def test_offsets_beyond_32_bits(cuda_device, kind):
    """Pages at the end of a cache of more than 2^32 elements (E4M3: bytes) and a block table whose rows are more than
    2^31 entries apart: append and decode give the bits of a small cache."""
    page, H, Hkv, lengths = 64, 16, 8, [200, 130]
    row = (Hkv, 128) if kind == "mha" else (576,)
    dtype = torch.uint8 if kind == "mla_fp8" else torch.bfloat16
    num = 2 ** 32 // (page * math.prod(row)) + 10
    # the table's rows lie in one buffer: entries 0.. and 2^31 + 16..
    wide = torch.empty(2 ** 31 + 32, dtype=torch.int32, device=DEV).as_strided((2, 4), (2 ** 31 + 16, 1))
    wide.copy_(torch.arange(num - 8, num, dtype=torch.int32).view(2, 4))
    near = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    sl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, lengths[0], sum(lengths)], dtype=torch.int32, device=DEV)
    T = sum(lengths)
    g = torch.Generator(device=DEV).manual_seed(7)
    rand = lambda *shape: torch.randn(*shape, dtype=torch.bfloat16, device=DEV, generator=g)
    cos_sin = M.rope_table(256, 128 if kind == "mha" else 64, device=DEV)
    k, v, q = rand(T, *((Hkv, 128) if kind == "mha" else (512,))), rand(T, *((Hkv, 128) if kind == "mha" else (64,))), \
        rand(2, 1, H, 128 if kind == "mha" else 576)
    results = []
    for table, pages in ((near, 8), (wide, num)):
        out, lse = blank(2, 1, H, 128 if kind == "mha" else 512)
        caches = [torch.empty(pages, page, *row, dtype=dtype, device=DEV) for _ in range(2 if kind == "mha" else 1)]
        if kind == "mha":
            plan = M.mha_decode_plan_paged(2, 1, H, Hkv, 256, page, device=0)
            ws = M.alloc_workspace(plan)
            M.mha_cache_append(k, v, cos_sin, *caches, table, sl, cu, workspace=ws)
            M.mha_decode_run_paged(plan, q, *caches, table, sl, 0.1, out, lse, ws)
        elif kind == "mla":
            plan = M.mla_decode_plan_paged(2, 1, H, 256, page, device=0)
            ws = M.alloc_workspace(plan)
            M.mla_cache_append(k, v, cos_sin, *caches, table, sl, cu, workspace=ws)
            M.mla_decode_run_paged(plan, q, *caches, table, sl, 0.05, out, lse, ws)
        else:
            plan = M.mla_decode_plan_paged_fp8(2, 1, H, 256, page, device=0)
            ws = M.alloc_workspace(plan)
            M.mla_cache_append(k, v, cos_sin, *caches, table, sl, cu, kv_scale=0.02, workspace=ws)
            M.mla_decode_run_paged_fp8(plan, q, *caches, 0.02, table, sl, 0.05, out, lse, ws)
        M.mla_decode_check(plan, ws)
        held = torch.cat([c[-8:].view(torch.uint8).view(2, 4 * page, -1)[b, :n] for c in caches for b, n in enumerate(lengths)])
        results.append((out, lse, held.clone()))
        del caches
    for small, large in zip(*results):
        assert torch.equal(small, large)
    assert bool(results[0][0].isfinite().all())


def test_tokens_with_the_same_place(cuda_device):
    """Two sequences that append to the same row of the same page: every element of it is one of theirs, and nothing else
    changes."""
    table = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    sl = torch.tensor([3, 3], dtype=torch.int32, device=DEV)
    x = torch.arange(1, 3, dtype=torch.bfloat16, device=DEV)[:, None].expand(2, 576).contiguous()
    angles = torch.cat([torch.ones(16, 32), torch.zeros(16, 32)], 1).to(DEV)  # no rotation
    kv = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    M.mla_cache_append(x[:, :512], x[:, 512:], angles, kv, table, sl)
    assert bool(((kv[0, 2] == 1) | (kv[0, 2] == 2)).all())
    kv[0, 2] = 0
    assert not bool(kv.any())
