"""Speculative decoding over caches that are kept small, as it is run: the drafted tokens' rows appended and their
queries brought into the cache's space, attention over each sequence's rows and its tree (the masks scattered from
lists of ancestors), the weights that the rows gather, the accepted tokens' rows appended again behind the cached ones,
the caches cut to a budget into fresh pages, and the next step over those.  Each operator's own tests hold it to
its definition; here the stages are held together, against 64 bits over the caches and queries that they left.

Tolerances: those of the operators' own tests, on the inputs that each stage had; of v_up as in the decode step's
test: what the attention's tolerance carries through |W|, and one more rounding.
"""

import numpy as np
import pytest
import torch

import token_sparse_mla_gb300 as smla
from tests import batch_reference as br
from tests import step_reference as ref
from tests.batch_reference import Batch
from tests.step_reference import base_fake, fake  # noqa: F401
from tests.test_evict import _kept
from tests.test_result_streams import BF, F32, I32, STREAM, CUDA0, _d, allocations  # noqa: F401
from types import SimpleNamespace
from workloads import make_v_up_weights

DEV = "cuda:0"


def _within(got, want, tol):
    assert np.all(np.abs(ref.to64(got) - want) <= tol), float((np.abs(ref.to64(got) - want) - tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("budget", [64, 150])
def test_gpu_verify_accept_evict_and_go_on(fmt, budget):
    seqs, h, dn = [(200, 7), (63, 12), (400, 1), (20, 5)], 16, 128
    new_blocks = -(-budget // 64) + 1
    batch = Batch(seqs, h, budget, fmt, spare=4 * new_blocks, pad=1)
    g = torch.Generator().manual_seed(1)
    T, B = batch.T, len(seqs)
    used = {int(p) for p in batch.tables.flatten() if p >= 0}
    free = torch.tensor([p for p in range(batch.cache.shape[0] // 64) if p not in used], dtype=torch.int32)
    new_tables = free[:B * new_blocks].reshape(B, new_blocks)
    table = ref.cos_sin_table(600)
    norm = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16)
    w_uk = (torch.randn(h, dn, 512, generator=g) * dn ** -0.5).to(torch.bfloat16)
    w_v = make_v_up_weights(h, 128, seed=4)
    scale = (dn + 64) ** -0.5
    d = {k: v.to(DEV) for k, v in dict(cache=batch.cache, tables=batch.tables, lengths=batch.lengths, starts=batch.starts, table=table,
                                       norm=norm, w_uk=w_uk, w_v=w_v, new_tables=new_tables).items()}

    def append(kv, positions, slots):
        smla.sparse_mla_append(kv.to(DEV), torch.tensor(positions, dtype=torch.int32, device=DEV),
                               torch.tensor(slots, dtype=torch.int32, device=DEV), d["cache"], d["table"], norm_weight=d["norm"], kv_format=fmt)

    # the drafted tokens: rows at their places behind the cached ones, queries turned by their depth in the tree
    kv = torch.randn(T, 576, generator=g).to(torch.bfloat16)
    positions, slots, lists = [-1] * T, [-1] * T, np.full((T, 12), -1, dtype=np.int32)
    for b, (n, k) in enumerate(seqs):
        at = batch.slots(b)
        for j in range(k):
            t = int(batch.starts[b]) + j
            above = np.nonzero(batch.sees[b][j])[0]
            positions[t], slots[t] = n + len(above) - 1, int(at[n + j])
            lists[t, :len(above)] = above
    append(kv, positions, slots)
    q_in = (torch.randn(T, h, dn + 64, generator=g) * 0.5).to(torch.bfloat16)
    q = smla.sparse_mla_q_up(q_in.to(DEV), d["w_uk"], torch.tensor(positions, dtype=torch.int32, device=DEV), d["table"])
    mask = smla.sparse_mla_scatter_mask(torch.from_numpy(lists).to(DEV), 12)
    out, lse = smla.sparse_mla_tree(q, d["cache"], d["tables"], d["lengths"], d["starts"], scale, mask=mask, kv_format=fmt)
    gathered = smla.sparse_mla_weights(q, d["cache"], d["tables"], d["lengths"], d["starts"], lse, scale, mask=mask, kv_format=fmt)
    y = smla.sparse_mla_v_up(out, d["w_v"])
    smla.sync_status()
    batch.cache, batch.q, batch.mask = d["cache"].cpu(), q.cpu(), mask.cpu()
    want_o, want_l, tol_o, tol_l = br.tree(batch, scale)
    live = slice(0, T - 1)
    _within(out[live], want_o[live], tol_o[live])
    _within(lse[live], want_l[live], tol_l[live])
    _within(gathered, *br.weights(batch, lse.cpu(), None, 1.0, scale))
    want_y = np.einsum("thk,hnk->thn", want_o[live], ref.to64(w_v))
    carried = np.einsum("thk,hnk->thn", tol_o[live], np.abs(ref.to64(w_v)))
    _within(y[live], want_y, carried * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want_y) + 1e-6)

    # a path of each tree is accepted: its rows once more, one behind the other
    accepted, lengths = [], []
    for b, (n, k) in enumerate(seqs):
        path = np.nonzero(batch.sees[b][k - 1])[0][:4]
        at = batch.slots(b)
        accepted += [(int(batch.starts[b]) + int(j), n + i, int(at[n + i])) for i, j in enumerate(path)]
        lengths.append(n + len(path))
    append(kv[[t for t, _, _ in accepted]], [p for _, p, _ in accepted], [s for _, _, s in accepted])
    smla.sync_status()
    after = d["cache"].cpu()
    for t, _, s in accepted:  # the same row as the drafted one was, at its new place
        assert torch.equal(after[s], batch.cache[slots[t]])

    # cut to the budget (as the weights of the drafted places stand), and one token more for each sequence
    d_len = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    kept, new_lengths, new_weights = smla.sparse_mla_evict(d["cache"], d["tables"], d_len, gathered, d["new_tables"], budget, sinks=2,
                                                           recent=8, kv_format=fmt)
    new_n = [min(n, budget) for n in lengths]
    assert new_lengths.tolist() == new_n
    for b, n in enumerate(lengths):
        mine = _kept(gathered[b].cpu().numpy(), n, budget, 2, 8)
        assert kept[b].tolist() == mine + [-1] * (budget - len(mine))
        assert torch.equal(new_weights[b, :len(mine)], gathered[b, mine])
    step = Batch([(n, 1) for n in new_n], h, 5, fmt, extra_blocks=4, tree="chain")
    step.blocks, step.tables = new_blocks, new_tables
    step_slots = [int(step.slots(b)[new_n[b]]) for b in range(B)]
    append(torch.randn(B, 576, generator=g).to(torch.bfloat16), lengths, step_slots)
    q2 = step.q.to(DEV)
    out2, lse2 = smla.sparse_mla_tree(q2, d["cache"], d["new_tables"], new_lengths, step.starts.to(DEV), scale, kv_format=fmt)
    weights2 = smla.sparse_mla_weights(q2, d["cache"], d["new_tables"], new_lengths, step.starts.to(DEV), lse2, scale, weights=new_weights,
                                       decay=0.5, out=new_weights.clone(), kv_format=fmt)
    smla.sync_status()
    step.cache = d["cache"].cpu()
    want_o, want_l, tol_o, tol_l = br.tree(step, scale)
    _within(out2, want_o, tol_o)
    _within(lse2, want_l, tol_l)
    _within(weights2, *br.weights(step, lse2.cpu(), new_weights.cpu(), 0.5, scale))


@pytest.mark.gpu
def test_gpu_tree_joins_with_a_shared_prefix():
    """The context in two parts: a prefix that all sequences share, and each one's own rows with its tree."""
    batch = Batch([(100, 6), (300, 2), (0, 9)], 16, 31)
    shared = torch.randperm(batch.cache.shape[0] // 64, generator=torch.Generator().manual_seed(2))[:3].int()
    batch.cache = torch.nan_to_num(batch.cache, 0.25)
    P, d = 170, batch.to(DEV)
    parts_o = torch.empty(2, batch.T, 16, 512, dtype=torch.bfloat16, device=DEV)
    parts_l = torch.empty(2, batch.T, 16, dtype=torch.float32, device=DEV)
    smla.sparse_mla_prefix(d["q"], d["kv_cache"], shared.to(DEV), P, out=parts_o[0], lse=parts_l[0])
    smla.sparse_mla_tree(**d, out=parts_o[1], lse=parts_l[1])
    out, lse = smla.sparse_mla_merge(parts_o, parts_l)
    smla.sync_status()
    at = np.arange(P)
    prefix = shared.numpy().astype(np.int64)[at // 64] * 64 + at % 64
    rows, q = batch.rows(), ref.to64(batch.q)
    for b in range(3):
        for t, slots, sees in batch.tokens(b):
            k = rows[np.concatenate([prefix, slots[sees]])]
            s = q[t] @ k.T * br.SCALE
            m = s.max(axis=1, keepdims=True)
            z = np.exp(s - m).sum(axis=1, keepdims=True)
            pr = np.exp(s - m) / z
            e = 576 * 2.0 ** -23 * br.SCALE * (np.abs(q[t]) @ np.abs(k).T).max(axis=1)
            # probabilities, each part's O and the merged O are rounded to bf16
            _within(out[t], pr @ k[:, :512], (3 * 2.0 ** -8 + 2 * e[:, None]) * (pr @ np.abs(k[:, :512])))
            want = (m + np.log(z))[:, 0]
            _within(lse[t], want, e + 2.0 ** -21 * np.abs(want) + 2.0 ** -19)


# ----------------------------------------------------------------------------- CPU: where results are allocated

def _calls():
    T, h = 3, 8
    q, kv, tables, lengths, starts = _d((T, h, 576), BF), _d((640, 576), BF), _d((2, 4), I32), _d((2,), I32), _d((3,), I32)
    return {
        "tree": (lambda **k: smla.sparse_mla_tree(q, kv, tables, lengths, starts, **k), 2, 1),
        "weights": (lambda **k: smla.sparse_mla_weights(q, kv, tables, lengths, starts, _d((T, h), F32), **k), 1, 0),
        "evict": (lambda **k: smla.sparse_mla_evict(kv, tables, lengths, _d((2, 256), F32), _d((2, 2), I32), 100, **k), 3, 0),
    }


@pytest.fixture
def asked(allocations, fake):  # noqa: F811
    from token_sparse_mla_gb300 import _binding
    _binding._tree_workspace_bytes.cache_clear()
    fake.lib.sparse_mla_tree_workspace_bytes = lambda *a: 1024
    yield allocations
    _binding._tree_workspace_bytes.cache_clear()


@pytest.mark.parametrize("name", list(_calls()))
@pytest.mark.parametrize("given,on", [(SimpleNamespace(device=CUDA0, cuda_stream=0x77E0), 0x77E0), (0x77E0, 0x77E0), (0, 0)])
def test_what_a_call_on_another_stream_allocates(asked, fake, name, given, on):  # noqa: F811
    call, results, scratch = _calls()[name]
    call(stream=given)
    assert [s for s, _, _ in asked] == [on] * (results + scratch)
    assert [r for _, _, r in asked] == [[STREAM]] * results + [[]] * scratch
    assert fake.lib.calls[-1][1][-1] == getattr(given, "cuda_stream", given)


@pytest.mark.parametrize("name", list(_calls()))
def test_what_a_call_on_the_current_stream_allocates(asked, name):
    call, results, scratch = _calls()[name]
    call()
    assert [(s, r) for s, _, r in asked] == [(STREAM, [])] * (results + scratch)
