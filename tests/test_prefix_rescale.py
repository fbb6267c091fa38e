"""sparse_mla_prefix where a piece has several blocks and a row's running max grows by more than 2^8
between them, so that the kernel rescales what it has accumulated.

The last rope dim sets the level of a page's logits (it is no part of the values): rows with +64 there
see it rise from block to block (or from page to page), rows with -64 see it fall, rows with 0 not move.

Tolerances as in test_prefix.py, with the sums over P keys counted: a logit is off by at most e = 576 *
2^-23 of its absolute sum; the fp32 sums of P terms by P * 2^-23 of theirs; O by 2^-8 of sum p |v| (p
rounded to bf16) and 2^-8 of itself.  A rescale is off by less than 2^-20, but what has been through it n
times weighs at most 2^-8n: under 2^-27 in all, less than a unit of the sums.
"""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import step_reference as ref
from tests.test_prefix import DEV, SCALE, _row_values, _run

LOG2E = 1.4426950408889634
# T, h, P: one piece of two or three blocks, also one that ends in page 0 or 1; 76 whole tiles; tiles cut
# into two pieces; pieces that cross into the next tile; more tiles than CTA pairs
SHAPES = [(1, 5, 200), (8, 16, 330), (9, 16, 384), (607, 16, 1000), (900, 4, 2500), (450, 8, 5100), (20, 512, 700)]


def _blocks_per_run(T, h, P):
    """At least this many blocks of 128 keys come one after another in a run of the kernel's plan, from
    the workspace that it asks for: none where every tile lies in one run, else two slots of partials a run."""
    rows, nblk = T * h, -(-P // 128)
    need = smla.prefix_workspace_bytes(T, h, P)
    if need == 0:
        return nblk
    runs = need // (2 * min(128, -(-rows // 32) * 32) * 514 * 4)
    return (-(-rows // 128) * nblk) // runs


@pytest.mark.parametrize("T,h,P", SHAPES)
def test_the_shapes_have_several_blocks_a_run(T, h, P):
    assert _blocks_per_run(T, h, P) >= 2


def _case(T, h, P, fmt, unit, seed):
    g = torch.Generator().manual_seed(seed)
    used = -(-P // 64)
    n = used + 2
    pages = torch.randperm(n, generator=g)[:used].int()
    q = (torch.randn(T * h, 576, generator=g) * 0.5).to(torch.bfloat16)
    at = torch.arange(T * h)
    # rows of a warp differ, and some warps have no row that grows
    q[:, 575] = torch.where(at // 32 % 4 == 2, -64.0, torch.where(at % 5 == 3, 0.0, 64.0)).to(torch.bfloat16)
    x = torch.randn(n * 64, 576, generator=g) * 0.5
    pos = torch.arange(P)
    slots = pages.long()[pos // 64] * 64 + pos % 64
    step = pos // (128 if unit == "block" else 64)
    x[slots, 575] = 2.5 * (step - int(step.max()) / 2.0)  # 6.7 in the logit, 2^9.6, a step
    live = torch.zeros(n * 64, dtype=torch.bool)
    live[slots] = True
    if fmt == "bf16":
        cache = x.to(torch.bfloat16)
        cache[~live] = float("nan")
    else:
        from workloads import quantize_fp8_rows
        cache = quantize_fp8_rows(x)
        cache[~live] = 0x7F
        cache[~live, 512:528] = 0xFF
    return q.reshape(T, h, 576), cache, pages


def _check(out, lse, q, cache, pages, P, fmt, skip=0):
    """skip: pages of the start that are masked.  Returns per row how often its max grew by 2^8."""
    rows = _row_values(cache, fmt)
    pos = torch.arange(skip * 64, P)
    k = rows[(pages.long()[pos // 64] * 64 + pos % 64).numpy()]
    x = ref.to64(q).reshape(-1, 576)
    s = (x @ k.T) * SCALE
    top = s.max(axis=1, keepdims=True)
    p = np.exp(s - top)
    z = p.sum(axis=1, keepdims=True)
    p /= z
    want_l, want_o, pv = (top + np.log(z))[:, 0], p @ k[:, :512], p @ np.abs(k[:, :512])
    e = 576 * 2.0 ** -23 * SCALE * (np.abs(x) @ np.abs(k).T).max(axis=1)
    sums = P * 2.0 ** -23
    assert np.all(np.abs(ref.to64(lse).reshape(-1) - want_l) <= e + sums + 2.0 ** -22 * np.abs(want_l) + 2.0 ** -20)
    tol = (2.0 ** -8 + 2 * e[:, None] + sums) * pv + 2.0 ** -8 * np.abs(want_o)
    err = np.abs(ref.to64(out).reshape(-1, 512) - want_o)
    assert np.all(err <= tol), float((err - tol).max())
    grown = np.zeros(len(x), dtype=int)
    m = np.full(len(x), -np.inf)
    for b in range(0, k.shape[0], 128):
        mx = s[:, b:b + 128].max(axis=1) * LOG2E
        grow = mx > m + 8.0
        grown += grow & np.isfinite(m)
        m = np.where(grow, mx, m)
    return grown


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("unit", ["block", "page"])
@pytest.mark.parametrize("T,h,P", SHAPES)
def test_gpu_max_that_grows_in_every_block(T, h, P, unit, fmt):
    assert _blocks_per_run(T, h, P) >= 2
    q, cache, pages = _case(T, h, P, fmt, unit, T + P)
    out, lse = _run(q, cache, pages, P, fmt)
    grown = _check(out, lse, q, cache, pages, P, fmt)
    rising = ref.to64(q).reshape(-1, 576)[:, 575] > 0
    assert np.all(grown[rising] == -(-P // 128) - 1) and np.all(grown[~rising] == 0)
    d = [x.to(DEV) for x in (q, cache, pages)]
    for _ in range(10):
        o, l = smla.sparse_mla_prefix(*d, P, kv_format=fmt)
        assert torch.equal(o.cpu(), out) and torch.equal(l.cpu(), lse)
    smla.sync_status()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T,h,P,skip", [(9, 16, 384, 2), (9, 16, 384, 3), (607, 16, 1000, 5), (450, 8, 5100, 33)])
def test_gpu_max_that_grows_after_masked_blocks(T, h, P, skip, fmt):
    """The first pages are outside the cache: a row's first max comes after blocks without a key."""
    q, cache, pages = _case(T, h, P, fmt, "block", T + P + 1)
    away = pages.clone()
    away[:skip] = -1
    out, lse = _run(q, cache, away, P, fmt)
    _check(out, lse, q, cache, pages, P, fmt, skip)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("P", [50, 128, 190, 256, 385])
def test_gpu_many_short_pieces_in_a_run(P, fmt):
    """300 tiles of one to four blocks: a CTA pair ends a piece and begins the next again and again, the
    accumulator read and then overwritten."""
    T, h = 600, 64
    q, cache, pages = _case(T, h, P, fmt, "page", P)
    out, lse = _run(q, cache, pages, P, fmt)
    _check(out, lse, q, cache, pages, P, fmt)
    d = [x.to(DEV) for x in (q, cache, pages)]
    for _ in range(3):
        o, l = smla.sparse_mla_prefix(*d, P, kv_format=fmt)
        assert torch.equal(o.cpu(), out) and torch.equal(l.cpu(), lse)
    smla.sync_status()
