"""A decode step as it is run: new rows appended to the cache, queries brought into its space, lists of
each sequence's own positions chosen, attention over the shared prefix and over the lists, merged, and
projected to values.  Each stage's own tests hold it to its definition; here the stages are held
together, against 64 bits over the cache and queries that the first two left.

Tolerance of the attention: the probabilities are rounded to bf16 (2^-8 of sum p |v|), each part's O
and the merged O are (2^-8 of sum p |v| each, which bounds |O|), and the logits' fp32 sums move the
probabilities by 2 e (576 * 2^-23 of the logit's absolute sum); of v_up: what that carries through |W|,
and one more rounding.
"""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import step_reference as ref
from tests.test_append import _check_rows
from tests.test_q_up import _check as check_q_up
from workloads import make_v_up_weights, quantize_fp8_rows

DEV = "cuda:0"


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("P,own,topk", [(200, 90, 48), (64, 3, 64), (1500, 130, 130)])
def test_gpu_decode_step(fmt, P, own, topk):
    T, h, dn, pad = 9, 16, 128, 2                     # two unused places at the end of the batch
    g = torch.Generator().manual_seed(P + own)
    live = T - pad
    shared_pages, own_pages = -(-P // 64), -(-(own + 1) // 64)
    perm = torch.randperm(shared_pages + T * own_pages + 2, generator=g).int()
    shared, mine = perm[:shared_pages].contiguous(), perm[shared_pages:shared_pages + T * own_pages].reshape(T, own_pages)
    n = perm.numel() * 64
    x = torch.randn(n, 576, generator=g) * 0.5
    cache = x.to(torch.bfloat16) if fmt == "bf16" else quantize_fp8_rows(x)

    # the new token of sequence t: own position `own`, absolute position P + own
    kv = torch.randn(T, 576, generator=g).to(torch.bfloat16)
    positions = torch.full((T,), P + own, dtype=torch.int32)
    slots = (mine[:, own // 64] * 64 + own % 64).int()
    positions[live:], slots[live:] = -1, -1
    norm = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16)
    table = ref.cos_sin_table(P + own + 1)
    q_in = (torch.randn(T, h, dn + 64, generator=g) * 0.5).to(torch.bfloat16)
    w = (torch.randn(h, dn, 512, generator=g) * dn ** -0.5).to(torch.bfloat16)
    w_v = make_v_up_weights(h, 128, seed=4)
    scores = torch.randn(T, own + 1, generator=g)
    lengths = torch.full((T,), own + 1, dtype=torch.int32)
    lengths[live:] = 0
    scale = (dn + 64) ** -0.5

    d = {k: v.to(DEV) for k, v in dict(kv=kv, positions=positions, slots=slots, norm=norm, table=table, q=q_in, w=w, w_v=w_v,
                                       scores=scores, lengths=lengths, shared=shared, cache=cache).items()}
    smla.sparse_mla_append(d["kv"], d["positions"], d["slots"], d["cache"], d["table"], norm_weight=d["norm"], kv_format=fmt)
    q = smla.sparse_mla_q_up(d["q"], d["w"], d["positions"], d["table"])
    lists = torch.empty(T, topk, dtype=torch.int32, device=DEV)
    for t in range(T):
        smla.sparse_mla_topk(d["scores"][t:t + 1], d["lengths"][t:t + 1], topk, block_table=mine[t].contiguous().to(DEV), out=lists[t:t + 1])
    parts_o = torch.empty(2, T, h, 512, dtype=torch.bfloat16, device=DEV)
    parts_l = torch.empty(2, T, h, dtype=torch.float32, device=DEV)
    smla.sparse_mla_prefix(q, d["cache"], d["shared"], P, scale, out=parts_o[0], lse=parts_l[0], kv_format=fmt)
    smla.sparse_mla_fwd(q, d["cache"], lists, scale, out=parts_o[1], lse=parts_l[1], kv_format=fmt)
    o, lse = smla.sparse_mla_merge(parts_o, parts_l)
    y = smla.sparse_mla_v_up(o, d["w_v"])
    smla.sync_status()

    _check_rows(cache, d["cache"], kv, positions, slots, table, norm, 1e-6, True, fmt)
    check_q_up(q.cpu(), q_in, w, positions, table, True)
    after = d["cache"].cpu()
    rows = ref.to64(after) if fmt == "bf16" else torch.from_numpy(ref.fp8_row_values(after)).float().to(torch.bfloat16).double().numpy()
    q64, wv64 = ref.to64(q), ref.to64(w_v)
    at = torch.arange(P)
    prefix_slots = (shared.long()[at // 64] * 64 + at % 64).numpy()
    for t in range(T):
        order = torch.argsort(scores[t, :int(lengths[t])], descending=True, stable=True)[:topk]
        own_slots = (mine[t].long()[order // 64] * 64 + order % 64).numpy()
        k = rows[np.concatenate([prefix_slots, own_slots])]
        if t < live:
            assert own in order.tolist() or topk < own + 1  # the new row takes part unless its score is too low
        s = np.einsum("hd,pd->hp", q64[t], k) * scale
        e = 576 * 2.0 ** -23 * scale * np.einsum("hd,pd->hp", np.abs(q64[t]), np.abs(k)).max(axis=1)
        m = s.max(axis=1, keepdims=True)
        z = np.exp(s - m).sum(axis=1, keepdims=True)
        p = np.exp(s - m) / z
        want_o, want_l = p @ k[:, :512], (m + np.log(z))[:, 0]
        tol = (3 * 2.0 ** -8 + 2 * e[:, None]) * (p @ np.abs(k[:, :512]))
        assert np.all(np.abs(ref.to64(lse)[t] - want_l) <= e + 2.0 ** -21 * np.abs(want_l) + 2.0 ** -19)
        assert np.all(np.abs(ref.to64(o)[t] - want_o) <= tol)
        want_y = np.einsum("hk,hnk->hn", want_o, wv64)
        carried = np.einsum("hk,hnk->hn", tol, np.abs(wv64))
        assert np.all(np.abs(ref.to64(y)[t] - want_y) <= carried * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want_y) + 1e-6)
