"""GPU tests of what the paged calls promise one another and their callers: an append behind a shared prefix turns by the
positions that the prefix's decode means, faults are told apart, arguments that would corrupt memory are refused.
Tolerances as in test_gpu_paged."""
import math

import pytest
import torch

from mla_decode_attention_11_b200 import binding as M
from tests.test_gpu_paged import (DEV, LONG, Pages, blank, close, make_prefix, make_window, rand, reference, seen_mask,
                                  turn_tolerance, turned)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [0, LONG])
@pytest.mark.parametrize("H", [16, 128])
def test_append_behind_a_prefix_then_decode(cuda_device, H, most):
    """A server's steps behind a system prompt that ends inside a page: the prompt is appended once, each sequence's own
    tokens with their own lengths, and the decode takes the same lengths.  Rows and queries are, bit for bit, those of
    whole sequences with the prompt in front, and the decode equals the 64-bit one over those; the step is captured and
    replayed after the prefix's length changed."""
    g = torch.Generator(device=DEV).manual_seed(4)
    page, P, prompts = 64, 100, [37, 0, 200, 64]
    B, total = len(prompts), [n + 3 for n in prompts]
    cos_sin, scale = M.rope_table(600, 64, device=DEV), 576 ** -0.5
    pages = Pages("mla", [*total, P], page, seed=5, width=-(-max(*total, most, P) // page))
    whole = Pages("mla", [P + n for n in total], page, seed=6)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    prefix_table, pl = pages.table[B].contiguous(), ints([P])
    prompt, row = rand(g, P, 576), rand(g, sum(prompts), 576)
    cu, sl = ints([0, *torch.tensor(prompts).cumsum(0).tolist()]), ints(prompts)
    M.mla_cache_append(prompt[:, :512], prompt[:, 512:], cos_sin, pages.k, prefix_table[None], ints([P]))
    M.mla_cache_append(row[:, :512], row[:, 512:], cos_sin, pages.k, pages.table[:B], sl, cu_tokens=cu, prefix_len=pl)
    # the whole sequences: the prompt, then the same rows
    each = prompt.repeat(B, 1)
    M.mla_cache_append(each[:, :512], each[:, 512:], cos_sin, whole.k, whole.table, ints([P] * B))
    M.mla_cache_append(row[:, :512], row[:, 512:], cos_sin, whole.k, whole.table, sl + P, cu_tokens=cu)
    plan = M.mla_decode_plan_prefix(B, 1, H, max(total), max(P, most), page, device=0)
    assert (plan.prefix_partitions > 0) == (most == LONG and H < 128)
    ws = M.alloc_workspace(plan)
    out, lse = blank(B, 1, H, 512)
    new, q_rope, q, q_whole = rand(g, B, 576), rand(g, B, H, 64), rand(g, B, H, 576), None

    def step():
        sl.add_(1)
        M.mla_cache_append(new[:, :512], new[:, 512:], cos_sin, pages.k, pages.table[:B], sl, q_rope=q_rope, q=q,
                           workspace=ws, prefix_len=pl)
        M.mla_decode_run_prefix(plan, q[:, None], pages.k, prefix_table, pl, pages.table[:B], sl, scale, out, lse, ws)

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
        q_whole = q.clone()
        q_whole[..., 512:] = 0
        M.mla_cache_append(new[:, :512], new[:, 512:], cos_sin, whole.k, whole.table, sl + P, q_rope=q_rope, q=q_whole)
        assert torch.equal(q, q_whole)
        want = turned(q_rope, cos_sin, sl.long() - 1 + P, True)
        assert ((q[..., 512:].double() - want).abs() <= turn_tolerance(q_rope, 64)(want)).all()
        seqs = [whole.double(whole.table[b], P + L) for b, L in enumerate(lengths)]
        for b, L in enumerate(lengths):
            held = torch.cat([pages.double(prefix_table, P)[0], pages.double(pages.table[b], L)[0]])
            assert torch.equal(held, seqs[b][0])
        reference.fp8 = 0.0
        masks = [seen_mask(P + L, 1, 0, 0) for L in lengths]
        close(out, lse, reference(q[:, None], seqs, masks, scale, None, 512), f"step {i}")
    # the captured step follows the prefix's length: 60 keys of it, the new tokens at positions 60 + p
    pl.fill_(60)
    sl.copy_(ints([n - 1 for n in total]))
    graph.replay()
    M.mla_decode_check(plan, ws)
    want = turned(q_rope, cos_sin, sl.long() - 1 + 60, True)
    assert ((q[..., 512:].double() - want).abs() <= turn_tolerance(q_rope, 64)(want)).all()
    assert sl.tolist() == total


def test_append_behind_a_prefix_flags(cuda_device):
    """Positions past the rotation table are skipped and reported; a negative prefix counts as none and is reported; a
    prefix of none is no prefix."""
    g = torch.Generator(device=DEV).manual_seed(1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    cos_sin, table, sl = M.rope_table(40, 64, device=DEV), ints([[1], [0]]), ints([10, 12])
    row, q_rope = rand(g, 4, 576), rand(g, 4, 16, 64)
    plan = M.mla_decode_plan_paged(2, 1, 16, 16, 16, device=0)
    ws = M.alloc_workspace(plan)

    def run(prefix, fp8=False, **kw):
        kv = torch.zeros(2, 16, 576, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV)
        q = torch.zeros(4, 16, 576, dtype=torch.bfloat16, device=DEV)
        M.mla_cache_append(row[:, :512], row[:, 512:], cos_sin, kv, table, sl, q_rope=q_rope, q=q, workspace=ws,
                           prefix_len=None if prefix is None else ints([prefix]), kv_scale=0.02 if fp8 else None, **kw)
        return kv, q

    for kw in (dict(), dict(interleaved=False), dict(fp8=True)):
        plain = run(None, **kw)
        none = run(0, **kw)
        M.mla_decode_check(plan, ws)
        assert all(torch.equal(x, y) for x, y in zip(plain, none))
        for bad in (-1, -2 ** 31):
            got = run(bad, **kw)
            with pytest.raises(M.MlaError) as e:
                M.mla_decode_check(plan, ws)
            assert e.value.code == 7 and all(torch.equal(x, y) for x, y in zip(plain, got))
    # 28 + 11 is the table's last position, 28 + 9 below it; one more is past it for the second sequence's last token
    run(28)
    M.mla_decode_check(plan, ws)
    kv, q = run(29)
    with pytest.raises(M.MlaError) as e:
        M.mla_decode_check(plan, ws)
    assert e.value.code == 7
    assert torch.count_nonzero(kv[0, 11]) == 0 and torch.count_nonzero(kv[0, 10]) > 0 and torch.count_nonzero(kv[1, 9]) > 0
    assert torch.count_nonzero(q[3]) == 0 and all(torch.count_nonzero(q[i]) > 0 for i in range(3))
    kv, q = run(2 ** 31 - 1)
    with pytest.raises(M.MlaError) as e:
        M.mla_decode_check(plan, ws)
    assert e.value.code == 7 and torch.count_nonzero(kv) == 0 and torch.count_nonzero(q) == 0
    for bad, error in ((ints([0, 0]), ValueError), (ints([0]).long(), TypeError), (ints([0]).cpu(), ValueError)):
        with pytest.raises(error):
            M.mla_cache_append(row[:, :512], row[:, 512:], cos_sin, kv, table, sl, prefix_len=bad)


@pytest.mark.parametrize("scale", [2.0 ** -149, 2.0 ** 126, 2.0 ** 127, 3e38, torch.finfo(torch.float32).max])
def test_append_takes_every_scale_of_fp32(cuda_device, scale):
    """Scales up to fp32's largest are positive and finite there; the codes are those of a division in 32 bits."""
    x = torch.arange(0, 65536, 16, device=DEV).to(torch.int32).to(torch.int16).view(torch.bfloat16).view(8, 512)
    x = torch.where(torch.isnan(x), 0.0, x)
    kv = torch.zeros(1, 16, 576, dtype=torch.uint8, device=DEV)
    table, sl = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([8], dtype=torch.int32, device=DEV)
    call = lambda s: M.mla_cache_append(x, torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV),
                                        M.rope_table(8, 64, device=DEV), kv, table, sl, kv_scale=s)
    call(scale)
    want = (x.float() / torch.tensor(scale, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert torch.equal(kv[0, :8, :512].contiguous().view(torch.float8_e4m3fn).float(), want)
    for bad in (2.0 ** 128, 3.5e38, math.inf):
        with pytest.raises(ValueError):
            call(bad)


@pytest.mark.parametrize("kind,H,Hkv", [("mla", 16, 1), ("mla", 128, 1), ("mla_fp8", 32, 1), ("mla_fp8", 128, 1),
                                        ("mha", 8, 2)])
def test_lengths_out_of_range_are_reported_as_such(cuda_device, kind, H, Hkv):
    """A length past L_max or below zero is clamped and reported as MLA_ERR_SEQLEN: where every table entry is good nothing
    else could be, and where pages are bad as well it comes first."""
    page, L_max, B = 64, 256, 3
    lengths = [100, 256, 30]
    run, _, (out, lse), (plan, ws, pages, sl, q) = make_window(kind, lengths, 1, H, Hkv, page, 0, 0, False, 19, L_max=L_max)
    # good pages everywhere: those of the second sequence, which is full
    pages.table.copy_(pages.table[1].expand(B, -1).clone())
    for bad, taken in ((L_max + 1, L_max), (2 ** 31 - 1, L_max), (-1, 0), (-2 ** 31, 0)):
        sl[0] = taken
        want = blank(*out.shape[:3], out.shape[3])
        run(*want)
        M.mla_decode_check(plan, ws)
        sl[0] = bad
        out.fill_(float("nan"))
        run(out, lse)
        with pytest.raises(M.MlaError) as e:
            M.mla_decode_check(plan, ws)
        assert e.value.code == 7, bad
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        M.mla_decode_check(plan, ws)  # reported once
    sl[0], pages.table[2, 0] = L_max + 1, -1
    run(out, lse)
    with pytest.raises(M.MlaError) as e:
        M.mla_decode_check(plan, ws)
    assert e.value.code == 7
    sl[0] = 100
    run(out, lse)
    with pytest.raises(M.MlaError) as e:
        M.mla_decode_check(plan, ws)
    assert e.value.code == 8


@pytest.mark.parametrize("most", [512, LONG])
@pytest.mark.parametrize("H", [16, 128])
def test_prefix_lengths_out_of_range_are_reported_as_such(cuda_device, H, most):
    """The same for the prefix's length, in both forms, and for the lengths behind a prefix."""
    run, _, (out, lse), (plan, ws, pages, sl, pl) = make_prefix([30, 0, 200], 1, H, 512, 64, False, seed=6, prefix_max=most,
                                                                L_max=256)
    # one good page for every entry of every table
    pages.k.nan_to_num_(0.5)
    pages.table.fill_(1)
    table = torch.ones(most // 64, dtype=torch.int32, device=DEV)
    B, scale = 3, 576 ** -0.5

    def call(o, l):
        M.mla_decode_run_prefix(plan, run.q, pages.k, table, pl, pages.table[:B], sl, scale, o, l, ws)
    for what, bad, taken in ((pl, most + 1, most), (pl, -5, 0), (sl[1:2], 257, 256), (sl[1:2], -1, 0)):
        keep = int(what)
        what.fill_(taken)
        want = blank(*out.shape[:3], 512)
        call(*want)
        M.mla_decode_check(plan, ws)
        what.fill_(bad)
        out.fill_(float("nan"))
        call(out, lse)
        with pytest.raises(M.MlaError) as e:
            M.mla_decode_check(plan, ws)
        assert e.value.code == 7, bad
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        what.fill_(keep)
