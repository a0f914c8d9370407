"""The softmax weights over E4M3 caches where they span many powers of two: a first token that outweighs thousands of
others together worth as much, scores that fall or rise tile after tile, heavy tails; contiguous and paged, both kernels
that multiply the codes themselves, a sequence in one piece and in several.

A score is one product: the query is zero but in a rope column (not a value column), so a key's score is its code there
times the head's query element, exactly, and a head's element sets how far the scores spread.  The 64-bit definition is
computed from the same codes.

Tolerances.  P is carried as two E4M3 terms: a weight is off by at most 2^-8 of itself (and 2^-11, as it passes through
f16), and by the terms' smallest step, whose sum over a sequence's keys the kernels hold below 2^-7 of the weights' sum.
The sums that normalise are of the weights themselves.  With A = sum p |v| / sum p and V = max |v|, out is off by
(2^-8 + 2^-11) A + 2^-7 V, and by 2^-8 of itself from its rounding.  Scores are fp32 products of exact factors: 2^-22 of
the largest |s| each, and lse 2^-20 (1 + |lse|) more.  The pieces' merge is fp32: 2^-20 A."""
import math

import pytest
import torch

from mla_decode_attention_11_b200 import binding as M

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
N = 30000


def profile(name, n, g):
    """[n] factors of the scores, at most 6.75 (448 / 64, E4M3's largest, is 7); the heads' query elements (in nats a unit)
    spread them."""
    j = torch.arange(n)
    x = torch.zeros(n)
    if name == "first":           # one key above all others, which are level
        x[0] = 1.0
    elif name == "first_noisy":   # the same, the others spread a little
        x = -0.02 * torch.randn(n, generator=g).abs()
        x[0] = 1.0
    elif name == "late":          # the dominant key comes last
        x[n - 1] = 1.0
    elif name == "every_tile":    # one in each tile
        x[::128] = 1.0
    elif name == "falling":       # down by a step every tile for 54 tiles, back to the top at the end
        x = -((j // 128).float() / 8).clamp(max=6.75)
        x[-100:] = 0.25
    elif name == "rising":
        x = ((j // 128).float() / 8).clamp(max=6.75)
    elif name == "levels":        # 128 keys at 1, 1000 at 1/2, the others at 0
        x[:128], x[128:1128] = 1.0, 0.5
    elif name == "tails":
        x = torch.randn(n, generator=g) / 4
    return x


def exact(q, k, v, L):
    s = q[:, None] * k[None, :L]                                     # [H, L]
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    return p @ v[:L], p @ v[:L].abs(), lse, s.abs().amax(1)


@pytest.mark.parametrize("name", ["first", "first_noisy", "late", "every_tile", "falling", "rising", "levels", "tails"])
@pytest.mark.parametrize("parts", [1, 7])
@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("paged", [False, True])
def test_weights_of_all_sizes(cuda_device, paged, H, parts, name):
    g = torch.Generator().manual_seed(11)
    page, ks = 64, 1.0 / 64
    L_max = -(-N // page) * page
    lengths = [N, 2047, 8192]
    codes = torch.zeros(len(lengths), L_max, 576)
    # values: a nonzero mean; the first key's are of the other sign, so that what it weighs shows
    codes[..., :512] = torch.randint(32, 97, (len(lengths), L_max, 512), generator=g).float()
    codes[:, 0, :512] = -64.0
    codes[:, :, 100:104] = 64.0                                      # constant columns: out = 1 whatever the weights
    for b, L in enumerate(lengths):
        codes[b, :L, 540] = profile(name, L, g) * 64
    codes = codes.to(torch.float8_e4m3fn)
    # the heads spread the scores by 6 to 14 nats a unit (steps of 1/16: exact in bf16 and in two E4M3 terms)
    spread = (6 + 8 * torch.arange(H) / H).mul(16).round().div(16)
    q = torch.zeros(len(lengths), 1, H, 576, dtype=torch.bfloat16)
    q[..., 540] = spread
    q, codes = q.to(DEV), codes.to(DEV)
    sl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    out = torch.full((len(lengths), 1, H, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(lengths), 1, H), float("nan"), dtype=torch.float32, device=DEV)
    if paged:
        plan = M.mla_decode_plan_paged_fp8(len(lengths), 1, H, L_max, page, device=0, num_partitions=parts)
        ws = M.alloc_workspace(plan)
        pages = codes.view(-1, page, 576)
        table = torch.arange(pages.shape[0], dtype=torch.int32, device=DEV).view(len(lengths), -1)
        M.mla_decode_run_paged_fp8(plan, q, pages, ks, table, sl, 1.0, out, lse, ws)
    else:
        plan = M.mla_decode_plan_fp8(len(lengths), 1, H, L_max, device=0, num_partitions=parts)
        ws = M.alloc_workspace(plan)
        M.mla_decode_run_fp8(plan, q, codes, ks, sl, 1.0, out, lse, ws)
    M.mla_decode_check(plan, ws)
    assert plan.kernel == (M.MLA_KERNEL_FP8_PAIR if H == 128 else M.MLA_KERNEL_FP8_MMA)
    for b, L in enumerate(lengths):
        kv = codes[b].double() * ks
        o, a, l, top = exact(spread.to(DEV).double(), kv[:, 540], kv[:, :512], L)
        weights = (2.0 ** -8 + 2.0 ** -11) * a + 2.0 ** -7 * kv[:L, :512].abs().max()
        delta = 2.0 ** -22 * top
        tol = weights + (2 * delta[:, None] + 2.0 ** -20) * a + 2.0 ** -8 * o.abs()
        err = (out[b, 0].double() - o).abs()
        assert torch.isfinite(out[b]).all()
        assert (err <= tol).all(), f"L {L}: out off by {err.max().item():.4f}, {(err / tol).max().item():.2f} tolerances"
        tol = delta + 2.0 ** -20 * (1 + l.abs())
        err = (lse[b, 0].double() - l).abs()
        assert (err <= tol).all(), f"L {L}: lse off by {err.max().item():.2e}, {(err / tol).max().item():.2f} tolerances"


@pytest.mark.parametrize("name", ["first", "first_noisy", "falling", "tails"])
@pytest.mark.parametrize("parts", [1, 7])
@pytest.mark.parametrize("H,Sq", [(16, 1), (16, 2), (64, 2), (128, 2)])
def test_first_tokens_and_a_window(cuda_device, H, Sq, parts, name):
    """The dominant key among the first tokens that stay visible, the others in a window of 9000: tiles of the first
    tokens, none in between, the window's; two query tokens see ranges one apart; sinks weigh too."""
    g = torch.Generator().manual_seed(12)
    page, ks, window, first = 16, 1.0 / 64, 9000, 4
    L_max = -(-N // page) * page
    lengths = [N, 8192, 1, 300]
    B = len(lengths)
    codes = torch.zeros(B, L_max, 576)
    codes[..., :512] = torch.randint(32, 97, (B, L_max, 512), generator=g).float()
    codes[:, :first, :512] = -64.0
    for b, L in enumerate(lengths):
        codes[b, :L, 540] = profile(name, L, g) * 64
    codes = codes.to(torch.float8_e4m3fn)
    spread = (6 + 8 * torch.arange(H) / H).mul(16).round().div(16)
    q = torch.zeros(B, Sq, H, 576, dtype=torch.bfloat16)
    q[..., 540] = spread
    sinks = torch.linspace(-3, 9, H)
    q, codes, sinks = q.to(DEV), codes.to(DEV), sinks.to(DEV)
    sl = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    out = torch.full((B, Sq, H, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, Sq, H), float("nan"), dtype=torch.float32, device=DEV)
    plan = M.mla_decode_plan_paged_fp8(B, Sq, H, L_max, page, window=window, first_tokens=first, device=0,
                                       num_partitions=parts)
    ws = M.alloc_workspace(plan)
    table = torch.arange(B * L_max // page, dtype=torch.int32, device=DEV).view(B, -1)
    M.mla_decode_run_paged_fp8(plan, q, codes.view(-1, page, 576), ks, table, sl, 1.0, out, lse, ws, sinks=sinks)
    M.mla_decode_check(plan, ws)
    for b, L in enumerate(lengths):
        kv = codes[b, :L].double() * ks
        for t in range(Sq):
            p = L - Sq + t
            j = torch.arange(L, device=DEV)
            seen = (j <= p) & ((j > p - window) | (j < first))
            s = torch.where(seen, spread.to(DEV).double()[:, None] * kv[:, 540], -math.inf)
            l = torch.logaddexp(torch.logsumexp(s, 1), sinks.double())
            w = torch.exp(s - l[:, None])
            o, a = w @ kv[:, :512], w @ kv[:, :512].abs()
            delta = 2.0 ** -22 * torch.where(seen, s.abs(), 0.0).amax(1)
            lost = 2.0 ** -7 * kv[:, :512].abs().max() * w.sum(1)[:, None]
            tol = (2.0 ** -8 + 2.0 ** -11 + 2 * delta[:, None] + 2.0 ** -20) * a + lost + 2.0 ** -8 * o.abs()
            err = (out[b, t].double() - o).abs()
            assert (err <= tol).all(), f"L {L} token {t}: out off by {err.max().item():.4f}"
            tol = delta + 2.0 ** -20 * (1 + l.abs())
            assert ((lse[b, t].double() - l).abs() <= tol).all(), f"L {L} token {t}: lse"
