"""sparse_mla_masked_mha where a row's running max grows by more than 2^8 in every tile of 64 keys, so that
O is rescaled in TMEM behind each PV, and where it falls or stays.

The last q/k dim sets a tile's level.  Tolerances, against 64 bits: a logit is off by at most e = dqk *
2^-23 of its absolute sum, the fp32 sums of S terms by S * 2^-23 of theirs, O by 2^-8 of sum p |v| (p
rounded to bf16) and 2^-8 of itself.  What a rescale (off by less than 2^-20) has touched n times weighs
at most 2^-8n: nothing beside these."""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests.step_reference import to64

DEV = "cuda:0"


def _case(T, S, h, dqk, dv, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(T, h, dqk, generator=g) * 0.5
    k = torch.randn(S, h, dqk, generator=g) * 0.5
    v = torch.randn(S, h, dv, generator=g)
    at = torch.arange(T)
    q[:, :, -1] = torch.where(at // 32 % 4 == 2, -64.0, torch.where(at % 5 == 3, 0.0, 64.0))[:, None]
    tile = torch.arange(S) // 64
    k[:, :, -1] = (1.75 * (tile - int(tile.max()) / 2.0))[:, None]
    bits = torch.rand(T, S, generator=g) < 0.8
    bits[:, ::64] = True  # every tile has a key for every row
    pad = torch.nn.functional.pad(bits, (0, -S % 32)).reshape(T, -1, 32).long()
    words = (pad << torch.arange(32)).sum(dim=2)
    mask = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int().contiguous()
    return q.to(torch.bfloat16), k.to(torch.bfloat16), v.to(torch.bfloat16), bits, mask


@pytest.mark.gpu
@pytest.mark.parametrize("dqk,dv", [(192, 128), (192, 256), (256, 128), (256, 256)])
@pytest.mark.parametrize("T,S,h", [(3, 150, 2), (300, 1500, 3), (129, 4100, 1), (2000, 500, 8)])
def test_gpu_max_that_grows_in_every_tile(T, S, h, dqk, dv):
    q, k, v, bits, mask = _case(T, S, h, dqk, dv, T + S + dqk)
    scale = dqk ** -0.5
    d = [x.to(DEV) for x in (q, k, v, mask)]
    out, lse = smla.sparse_mla_masked_mha(*d, scale)
    smla.sync_status()
    keep = bits.numpy()
    for hh in range(h):
        qq, kk, vv = to64(q[:, hh]), to64(k[:, hh]), to64(v[:, hh])
        s = np.where(keep, qq @ kk.T * scale, -np.inf)
        top = s.max(axis=1, keepdims=True)
        p = np.exp(s - top)
        z = p.sum(axis=1, keepdims=True)
        p /= z
        want_l, want_o = (top + np.log(z))[:, 0], p @ vv
        e = dqk * 2.0 ** -23 * scale * (np.abs(qq) @ np.abs(kk).T).max(axis=1)
        sums = S * 2.0 ** -23
        assert np.all(np.abs(to64(lse[:, hh]) - want_l) <= e + sums + 2.0 ** -22 * np.abs(want_l) + 2.0 ** -20)
        tol = (2.0 ** -8 + 2 * e[:, None] + sums) * (p @ np.abs(vv)) + 2.0 ** -8 * np.abs(want_o)
        assert np.all(np.abs(to64(out[:, hh]) - want_o) <= tol)
        # the rows with +64 are rescaled behind every tile, the others never
        tops = np.stack([s[:, b:b + 64].max(axis=1) for b in range(0, S, 64)], axis=1) * np.log2(np.e)
        rising = qq[:, -1] > 0
        assert np.all(np.diff(tops[rising], axis=1) > 8.0) and np.all(np.diff(tops[~rising], axis=1) < 8.0)
    for _ in range(10):
        o, l = smla.sparse_mla_masked_mha(*d, scale)
        assert torch.equal(o, out) and torch.equal(l, lse)
    smla.sync_status()


def test_the_inputs_grow_as_described():
    for dqk in (192, 256):
        q, k, _, bits, _ = _case(300, 1500, 1, dqk, 128, 7)
        s = np.where(bits.numpy(), to64(q[:, 0]) @ to64(k[:, 0]).T * dqk ** -0.5, -np.inf)
        tops = np.stack([s[:, b:b + 64].max(axis=1) for b in range(0, 1500, 64)], axis=1) * np.log2(np.e)
        rising = to64(q[:, 0])[:, -1] > 0
        assert np.all(np.diff(tops[rising], axis=1) > 8.0) and np.all(np.diff(tops[~rising], axis=1) < 8.0)
