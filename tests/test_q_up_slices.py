"""sparse_mla_q_up where a CTA has many (head, token tile) items: slices of 256 latent dims (192 nope
dims, from as many items as fill the SMs), the last item count below them, and runs that cross from a head
into the next one.  Tolerances as in test_q_up.py."""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import step_reference as ref
from tests.test_q_up import DEV, _case


def _definition(q, w, pos, table, interleaved):
    """q_up in 64 bits, and the absolute sums that its tolerances take."""
    x, ww, tab = ref.to64(q), ref.to64(w), ref.to64(table)
    dn = ww.shape[1]
    nope, rope = x[:, :, :dn].transpose(1, 0, 2), x[:, :, dn:]
    latent = (nope @ ww).transpose(1, 0, 2)
    absum = (np.abs(nope) @ np.abs(ww)).transpose(1, 0, 2)
    at = pos.long().numpy()
    cos, sin = tab[at, None, :32], tab[at, None, 32:]
    if interleaved:
        a, b = rope[..., 0::2], rope[..., 1::2]
    else:
        a, b = rope[..., :32], rope[..., 32:]
    y0, y1, size = a * cos - b * sin, b * cos + a * sin, np.abs(a) + np.abs(b)
    if interleaved:
        turned, size = np.stack([y0, y1], -1).reshape(rope.shape), np.repeat(size, 2, axis=-1)
    else:
        turned, size = np.concatenate([y0, y1], -1), np.concatenate([size, size], -1)
    return latent, absum, turned, size


def test_the_definition_is_the_other_one():
    """Two plain forms, written apart."""
    for interleaved in (True, False):
        q, w, pos, table = _case(5, 3, 128, 2)
        latent, _, turned, _ = _definition(q, w, pos, table, interleaved)
        want = ref.q_up(q, w, pos, table, interleaved)
        assert np.allclose(latent, want[:, :, :512], rtol=1e-12, atol=1e-12) and np.allclose(turned, want[:, :, 512:], rtol=1e-12, atol=0)


# 152 SMs: 256-dim slices from 76 items on
@pytest.mark.gpu
@pytest.mark.parametrize("T,h,dn,interleaved", [
    (1001, 64, 192, True), (1001, 64, 192, False),    # 512 items: seven a CTA, heads change inside most runs
    (257, 40, 192, True), (257, 40, 192, False),      # three tiles a head, the last of one token
    (3900, 3, 192, False), (3900, 3, 192, True),      # 31 tiles a head, a head changes inside a few runs
    (76 * 128, 1, 192, True), (75 * 128, 1, 192, True),  # at the threshold and one item below
    (38 * 128 - 1, 2, 192, False), (1, 76, 192, False), (1, 75, 192, False),
    (257, 40, 256, True), (257, 40, 256, False), (257, 40, 128, False)])
def test_gpu_many_items(T, h, dn, interleaved):
    q, w, pos, table = _case(T, h, dn, T + h)
    guard = torch.full((T + 2, h, 576), 3.5, dtype=torch.bfloat16, device=DEV)
    d = [x.to(DEV) for x in (q, w, pos, table)]
    out = smla.sparse_mla_q_up(*d, interleaved=interleaved, out=guard[1:T + 1])
    smla.sync_status()
    latent, absum, turned, size = _definition(q, w, pos, table, interleaved)
    got = ref.to64(out)
    tol = 2.0 ** -8 * np.abs(latent) * (1 + 2.0 ** -10) + dn * 2.0 ** -23 * absum
    assert np.all(np.abs(got[:, :, :512] - latent) <= tol)
    tol = 2.0 ** -8 * np.abs(turned) * (1 + 2.0 ** -10) + 4 * 2.0 ** -24 * size
    assert np.all(np.abs(got[:, :, 512:] - turned) <= tol)
    assert guard[0].eq(3.5).all() and guard[T + 1].eq(3.5).all()
    for _ in range(5):
        assert torch.equal(smla.sparse_mla_q_up(*d, interleaved=interleaved), out)
    smla.sync_status()
