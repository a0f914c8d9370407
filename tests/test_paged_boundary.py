"""The paged cache's C ABI on the CPU: plans, refusals before anything is launched, the binding's structures, and the
rotation table."""
import ctypes
import math
import os
import re

import pytest
import torch

from mla_decode_attention_11_b200 import binding as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCALE = ctypes.c_float(0.04)


@pytest.fixture(scope="module")
def lib():
    return M.load_library()


def test_plans():
    p = M.mla_decode_plan_paged(4, 1, 128, 5000, 64, window=1000, first_tokens=4, device=-1)
    assert (p.kernel, p.page_size, p.window, p.first_tokens) == (M.MLA_KERNEL_PAIR, 64, 1000, 4)
    assert p.workspace_bytes == M.mla_decode_plan(4, 1, 128, 5000, device=-1).workspace_bytes
    assert M.mla_decode_plan_paged(4, 1, 16, 5000, 16, device=-1).kernel == M.MLA_KERNEL_TRANSPOSED
    assert M.mla_decode_plan_paged_fp8(4, 1, 128, 5000, 16, device=-1).kernel == M.MLA_KERNEL_FP8_PAIR
    assert M.mla_decode_plan_paged_fp8(4, 1, 16, 5000, 64, device=-1).kernel == M.MLA_KERNEL_FP8_MMA
    assert M.mha_decode_plan_paged(4, 1, 32, 8, 5000, 16, device=-1).kernel == M.MLA_KERNEL_MHA
    # few heads and much to read: a launch of its own for the prefix, 160 rows in two groups of 128
    p = M.mla_decode_plan_prefix(5, 2, 16, 100, 90000, 48, device=-1)
    assert (p.prefix_max, p.prefix_groups, p.prefix_partitions, p.page_size) == (90000, 2, 74, 48)
    # one fp32 partial a query row for the prefix and one for its own keys
    assert p.workspace_bytes >= (p.prefix_groups * 128 + 160) * 513 * 4
    # else the prefix is read in front of every sequence's keys, in one launch
    for args in ((5, 2, 16, 100, 9000, 48), (64, 1, 128, 1000, 1 << 20, 64)):
        p = M.mla_decode_plan_prefix(*args, device=-1)
        assert p.prefix_groups == p.prefix_partitions == 0
        assert p.workspace_bytes == M.mla_decode_plan(*args[:4], device=-1).workspace_bytes


@pytest.mark.parametrize("page,window,first,code", [
    (0, 0, 0, 1), (-16, 0, 0, 1), (8, 0, 0, 3), (40, 0, 0, 3), ((1 << 24) + 16, 0, 0, 1), (16, -1, 0, 1),
    (16, 1, -1, 1), (16, 1, (1 << 24) + 1, 1)])
def test_plans_reject(page, window, first, code):
    for make in (lambda: M.mla_decode_plan_paged(2, 1, 16, 100, page, window, first, device=-1),
                 lambda: M.mla_decode_plan_paged_fp8(2, 1, 16, 100, page, window, first, device=-1),
                 lambda: M.mha_decode_plan_paged(2, 1, 8, 2, 100, page, window, first, device=-1)):
        with pytest.raises(M.MlaError) as e:
            make()
        assert e.value.code == code


def test_prefix_plan_rejects():
    for args, code in (((2, 1, 16, 100, 0, 16), 1), ((2, 1, 16, 100, (1 << 24) + 1, 16), 1),
                       ((2, 1, 16, 100, 10, 24), 3), ((2, 1, 24, 100, 10, 16), 3), ((0, 1, 16, 100, 10, 16), 1)):
        with pytest.raises(M.MlaError) as e:
            M.mla_decode_plan_prefix(*args, device=-1)
        assert e.value.code == code


def run_args(plan, **kw):
    a = dict(q=16, kv=16, pages=10, table=16, stride=8, width=8, sl=16, sinks=None, out=16, lse=16, ws=256,
             bytes=plan.workspace_bytes)
    a.update(kw)
    return a


def test_run_rejects_without_launching(lib):
    mla = M.mla_decode_plan_paged(2, 1, 16, 128, 16, device=-1)
    fp8 = M.mla_decode_plan_paged_fp8(2, 1, 16, 128, 16, device=-1)
    mha = M.mha_decode_plan_paged(2, 1, 8, 2, 128, 16, device=-1)
    pre = M.mla_decode_plan_prefix(2, 1, 16, 128, 128, 16, device=-1)
    flat = M.mla_decode_plan(2, 1, 16, 128, device=-1)

    def call(kind, plan, kv_scale=0.5, pt=16, pw=8, pl=16, **kw):
        a = run_args(plan, **kw)
        tail = (a["table"], a["stride"], a["width"], a["sl"], SCALE, a["sinks"], a["out"], a["lse"], a["ws"], a["bytes"],
                None)
        ref = ctypes.byref(plan)
        if kind == "mla":
            return lib.mla_decode_run_paged(ref, a["q"], a["kv"], a["pages"], *tail)
        if kind == "fp8":
            return lib.mla_decode_run_paged_fp8(ref, a["q"], a["kv"], a["pages"], ctypes.c_float(kv_scale), *tail)
        if kind == "mha":
            return lib.mha_decode_run_paged(ref, a["q"], a["kv"], a["kv"], a["pages"], *tail)
        return lib.mla_decode_run_prefix(ref, a["q"], a["kv"], a["pages"], pt, pw, pl, *tail)

    plans = {"mla": mla, "fp8": fp8, "mha": mha, "pre": pre}
    for kind, plan in plans.items():
        for bad in (dict(q=None), dict(kv=None), dict(table=None), dict(sl=None), dict(out=None), dict(lse=None),
                    dict(pages=0), dict(stride=-1), dict(width=7), dict(width=0)):
            assert call(kind, plan, **bad) == 1, (kind, bad)
        for bad in (dict(q=24), dict(kv=8), dict(table=18), dict(sl=17), dict(out=20), dict(lse=18), dict(sinks=18)):
            assert call(kind, plan, **bad) == 2, (kind, bad)
        for bad in (dict(ws=None), dict(ws=128), dict(bytes=plan.workspace_bytes - 1)):
            assert call(kind, plan, **bad) == 6, (kind, bad)
        for other, p in {**plans, "flat": flat}.items():
            if other != kind:
                assert call(kind, p) == 1, (kind, other)
    for bad in (0.0, -1.0, math.nan, math.inf):
        assert call("fp8", fp8, kv_scale=bad) == 1
    assert call("pre", pre, pt=None) == 1 and call("pre", pre, pl=None) == 1 and call("pre", pre, pw=7) == 1
    assert call("pre", pre, pt=18) == 2 and call("pre", pre, pl=18) == 2
    # the contiguous entry points refuse paged plans
    a = run_args(mla)
    assert lib.mla_decode_run(ctypes.byref(mla), 16, 16, 16, SCALE, 16, 16, 256, a["bytes"], None) == 1
    assert lib.mla_decode_run_noalloc(ctypes.byref(mla), 16, 16, 16, SCALE, 16, 16, 0, None) == 1
    assert lib.mla_decode_run_fp8(ctypes.byref(fp8), 16, 16, SCALE, 16, SCALE, None, 16, 16, 256,
                                  fp8.workspace_bytes, None) == 1
    assert lib.mha_decode_run(ctypes.byref(mha), 16, 16, 16, 16, SCALE, None, 16, 16, 256, mha.workspace_bytes,
                              None) == 1


FIELDS = ("B T H Hkv rope_dim interleaved num_positions page_size num_pages table_width table_stride cu_tokens seqlens "
          "block_table cos_sin k v q_in q_out k_pages v_pages k_token_stride k_head_stride v_token_stride v_head_stride "
          "q_in_token_stride q_in_head_stride q_out_token_stride q_out_head_stride status kv_scale reserved").split()


def test_append_fields_match_the_header():
    """The binding packs mla_append's fields in the header's order."""
    text = open(os.path.join(ROOT, "include", "mla_decode.h")).read()
    body = re.search(r"typedef struct mla_append \{(.*?)\} mla_append;", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n.strip(" *") for decl in body.split(";") if decl.strip()
             for n in re.sub(r"^\s*(const\s+)?\w+\s+", "", decl.strip()).split(",")]
    assert [n.replace("const ", "").split()[-1].strip("*") for n in names] == FIELDS
    assert M._APPEND.size == 4 * 10 + 8 * 20 + 8


def append(lib, kind, **kw):
    a = dict(B=2, T=4, H=0, Hkv=2, rope_dim=64, interleaved=0, num_positions=100, page_size=16, num_pages=4,
             table_width=4, table_stride=4, cu_tokens=16, seqlens=16, block_table=16, cos_sin=16, k=16, v=16, q_in=0,
             q_out=0, k_pages=16, v_pages=16, k_token_stride=512, k_head_stride=0, v_token_stride=64, v_head_stride=0,
             q_in_token_stride=0, q_in_head_stride=0, q_out_token_stride=0, q_out_head_stride=0, status=0, kv_scale=0.0,
             reserved=0)
    assert set(kw) <= set(a)
    a.update(kw)
    fn = lib.mla_cache_append if kind == "mla" else lib.mha_cache_append
    return fn(M._APPEND.pack(*(a[f] for f in FIELDS)), None)


@pytest.mark.parametrize("kind", ["mla", "mha"])
def test_append_rejects_without_launching(lib, kind):
    for bad in (dict(B=0), dict(T=-1), dict(H=-1), dict(H=70000, q_in=16, q_out=16), dict(page_size=0),
                dict(num_pages=0), dict(table_width=0), dict(table_stride=-1), dict(num_positions=0),
                dict(interleaved=2), dict(cu_tokens=0, T=3), dict(seqlens=0), dict(block_table=0), dict(cos_sin=0),
                dict(k=0), dict(v=0), dict(k_pages=0), dict(H=4), dict(H=4, q_in=16), dict(kv_scale=-1.0),
                dict(kv_scale=math.nan), dict(kv_scale=math.inf), dict(rope_dim=0), dict(rope_dim=72)):
        assert append(lib, kind, **bad) == 1, bad
    for bad in (dict(k=24), dict(v=8), dict(k_pages=8), dict(cos_sin=8), dict(seqlens=18), dict(cu_tokens=18),
                dict(block_table=18), dict(status=18), dict(k_token_stride=516), dict(v_token_stride=1),
                dict(H=4, q_in=24, q_out=16), dict(H=4, q_in=16, q_out=24),
                dict(H=4, q_in=16, q_out=16, q_out_head_stride=100)):
        assert append(lib, kind, **bad) == 2, bad
    if kind == "mla":
        assert append(lib, kind, rope_dim=128) == 1
    else:
        for bad in (dict(v_pages=0), dict(Hkv=0), dict(rope_dim=144), dict(kv_scale=0.5)):
            assert append(lib, kind, **bad) == 1, bad
    assert append(lib, kind, T=0, k=0, v=0, H=4) == 0  # nothing to do


def test_host_tensors_are_refused():
    plan = M.mla_decode_plan_paged(1, 1, 16, 16, 16, device=-1)
    q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16)
    kv, i = torch.zeros(1, 16, 576, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.mla_decode_run_paged(plan, q, kv, i, i[0], 0.04, q[..., :512], q[..., 0], kv)
    row = torch.zeros(1, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        M.mla_cache_append(row[:, :512], row[:, 512:], M.rope_table(4, 64), kv, i, i[0])


@pytest.mark.parametrize("dim,base", [(64, 10000.0), (128, 500000.0)])
def test_rope_table(dim, base):
    t = M.rope_table(30000, dim, base)
    assert t.shape == (30000, dim) and t.dtype == torch.float32
    for p in (0, 1, 777, 29999):
        for i in (0, 1, dim // 2 - 1):
            angle = p * base ** (-2 * i / dim)
            # 64-bit angles (their error times p), then half a step of fp32
            assert abs(float(t[p, i]) - math.cos(angle)) <= 2.0 ** -24 + p * 2.0 ** -50
            assert abs(float(t[p, dim // 2 + i]) - math.sin(angle)) <= 2.0 ** -24 + p * 2.0 ** -50


def test_status_names():
    assert M.STATUS_NAMES[8] == "MLA_ERR_PAGE" and M.status_string(8)
