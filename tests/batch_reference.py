"""Plain 64-bit forms of the operators on a batch of sequences (tree attention, gathered weights, eviction),
written from their definitions in include/sparse_mla.h (CPU, numpy; no code of the library), and the
batches that their tests share."""

import numpy as np
import torch

from tests import step_reference as ref

SCALE = 576 ** -0.5


class Batch:
    """Sequences of (cached rows, drafted tokens): their tables, lengths, starts, cache, queries and masks.
    Every cache row that is no position of a sequence holds NaN (`dead` says other bits)."""

    def __init__(self, seqs, h, seed, fmt="bf16", *, q_sd=1.0, pad=0, lead=0, spare=3, extra_blocks=0, tree="random", words=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.seqs, self.h, self.fmt = list(seqs), h, fmt
        self.T = lead + sum(d for _, d in seqs) + pad
        self.blocks = max([1] + [-(-(n + d) // 64) for n, d in seqs]) + extra_blocks
        used = [-(-(n + d) // 64) for n, d in seqs]
        pages = sum(used) + spare
        perm = torch.randperm(pages, generator=g)
        self.tables = torch.full((len(seqs), self.blocks), -7, dtype=torch.int32)
        live = torch.zeros(pages * 64, dtype=torch.bool)
        at = 0
        for b, (n, d) in enumerate(seqs):
            self.tables[b, :used[b]] = perm[at:at + used[b]].int()
            at += used[b]
            if n + d:
                live[self.slots(b)] = True
        self.lengths = torch.tensor([n for n, _ in seqs], dtype=torch.int32)
        self.starts = torch.tensor(np.cumsum([lead] + [d for _, d in seqs]), dtype=torch.int32)
        x = torch.randn(pages * 64, 576, generator=g) * 0.5
        if fmt == "bf16":
            self.cache = x.to(torch.bfloat16)
            self.cache[~live] = float("nan")
        else:
            from workloads import quantize_fp8_rows
            self.cache = quantize_fp8_rows(x)
            self.cache[~live] = 0x7F
            self.cache[~live, 512:528] = 0xFF
        self.q = (torch.randn(self.T, h, 576, generator=g) * q_sd).to(torch.bfloat16)
        most = max([1] + [d for _, d in seqs])
        self.words = words or -(-most // 32)
        self.sees = []  # per sequence [tokens, drafted]
        for _, d in seqs:
            m = np.zeros((d, d), dtype=bool)
            for j in range(d):
                if tree == "random":
                    if j:
                        m[j] = m[rng.integers(max(0, j - 8), j)]
                    m[j, j] = True
                elif tree == "chain":
                    m[j, :j + 1] = True
                elif tree == "any":
                    m[j] = rng.random(d) < 0.4
            self.sees.append(m)
        self.mask = None if tree == "chain" else self.pack()

    def pack(self):
        mask = np.full((self.T, self.words), 0xFFFFFFFF, dtype=np.uint32)  # of no sequence: anything
        for b, m in enumerate(self.sees):
            for j in range(m.shape[0]):
                bits = np.zeros(self.words * 32, dtype=np.uint64)
                k = min(m.shape[1], bits.size)
                bits[:k] = m[j, :k]
                bits[m.shape[1]:] = 1  # bits past the last drafted token: nobody there
                mask[int(self.starts[b]) + j] = (bits.reshape(-1, 32) << np.arange(32, dtype=np.uint64)).sum(axis=1).astype(np.uint32)
        return torch.from_numpy(mask.view(np.int32).copy())

    def slots(self, b):
        """Slots of the positions of sequence b (numpy int64), -1 where the table names no page of a cache."""
        n, d = self.seqs[b]
        at = np.arange(min(n + d, self.blocks * 64))
        page = self.tables[b].numpy().astype(np.int64)[at // 64]
        return np.where(page >= 0, page * 64 + at % 64, -1)

    def rows(self):
        """fp64 values of all cache rows as the kernels multiply them."""
        if self.fmt == "bf16":
            return ref.to64(self.cache)
        with np.errstate(all="ignore"):
            return torch.from_numpy(ref.fp8_row_values(self.cache)).float().to(torch.bfloat16).double().numpy()

    def tokens(self, b):
        """(token, its sequence's slots, which of them it sees) of sequence b; slots outside the cache are seen by none."""
        n, d = self.seqs[b]
        slots = self.slots(b)
        inside = (slots >= 0) & (slots < self.cache.shape[0])
        for j in range(d):
            sees = np.concatenate([np.ones(n, dtype=bool), self.sees[b][j]])[:slots.size]
            if self.mask is not None:
                sees[n + 32 * self.words:] = False
            yield int(self.starts[b]) + j, slots, sees & inside

    def to(self, dev):
        return dict(q=self.q.to(dev), kv_cache=self.cache.to(dev), block_tables=self.tables.to(dev), lengths=self.lengths.to(dev),
                    starts=self.starts.to(dev), mask=None if self.mask is None else self.mask.to(dev))


def tree(batch, scale=SCALE):
    """out [T, h, 512], lse [T, h] in fp64 and their tolerances (NaN rows of no sequence), by the arithmetic of
    tests/test_tree.py."""
    rows, q = batch.rows(), ref.to64(batch.q)
    out, lse = np.full((batch.T, batch.h, 512), np.nan), np.full((batch.T, batch.h), np.nan)
    tol_o, tol_l = np.zeros_like(out), np.zeros_like(lse)
    for b in range(len(batch.seqs)):
        for t, slots, sees in batch.tokens(b):
            k = rows[slots[sees]]
            if not len(k):
                out[t], lse[t] = 0, -np.inf
                continue
            s = (q[t] @ k.T) * scale
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(axis=1, keepdims=True)
            p = e / z
            out[t], lse[t] = p @ k[:, :512], (m + np.log(z))[:, 0]
            err = 576 * 2.0 ** -23 * abs(scale) * (np.abs(q[t]) @ np.abs(k).T).max(axis=1)
            tol_l[t] = err + 2.0 ** -22 * np.abs(lse[t]) + 2.0 ** -20
            tol_o[t] = (2.0 ** -8 + 2 * err[:, None]) * (p @ np.abs(k[:, :512])) + 2.0 ** -8 * np.abs(out[t]) + 1e-30
    return out, lse, tol_o, tol_l


def weights(batch, lse, prev, decay, scale=SCALE):
    """out [seqs, blocks * 64] in fp64 and its tolerance, by the arithmetic of tests/test_weights.py; lse [T, h] fp32."""
    rows, q, lse = batch.rows(), ref.to64(batch.q), ref.to64(lse)
    width = batch.blocks * 64
    out, tol = np.zeros((len(batch.seqs), width)), np.zeros((len(batch.seqs), width))
    for b, (n, d) in enumerate(batch.seqs):
        n = min(n, width)
        if prev is not None:
            out[b, :n] = decay * ref.to64(prev)[b, :n]
        for t, slots, sees in batch.tokens(b):
            at = np.nonzero(sees)[0]
            k = rows[slots[at]]
            fin = ~np.isneginf(lse[t])
            y = (q[t][fin] @ k.T) * scale - lse[t][fin, None]
            p = np.exp(y)
            err = 576 * 2.0 ** -23 * abs(scale) * (np.abs(q[t][fin]) @ np.abs(k).T)
            out[b, at] += p.sum(axis=0)
            tol[b, at] += (p * (np.expm1(err + np.abs(y) * 2.0 ** -23) + 2.0 ** -22)).sum(axis=0)
        tol[b] += (d * batch.h + 3) * 2.0 ** -24 * np.abs(out[b])
    return out, tol
