"""Plain 64-bit forms of the operators around the attention (append, q_up, prefix), written from
their definitions in include/sparse_mla.h (CPU, numpy; no code of the library), and what their
tests share."""

import numpy as np
import pytest
import torch

from tests import test_binding_marshal as marshal
from token_sparse_mla_gb300 import _binding

CUDA0, STREAM, _d = marshal.CUDA0, marshal.STREAM, marshal._d
base_fake = marshal.fake


@pytest.fixture
def fake(base_fake, monkeypatch):
    """The recording library of the marshalling tests, with the raw handle of the current stream."""
    monkeypatch.setattr(_binding, "_current_handle", lambda dev: STREAM)
    _binding._prefix_workspace_bytes.cache_clear()
    yield base_fake
    _binding._prefix_workspace_bytes.cache_clear()


def to64(x: torch.Tensor) -> np.ndarray:
    """bf16 / fp32 -> fp64, exact."""
    return x.detach().cpu().double().numpy()


def cos_sin_table(max_pos: int, base: float = 10000.0) -> torch.Tensor:
    """[max_pos, 64] fp32: 32 cosines, then 32 sines of position * base^(-i / 32)."""
    ang = np.arange(max_pos)[:, None] * base ** (-np.arange(32) / 32.0)[None, :]
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32))


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """One vector of 64 values, its 32 pairs turned."""
    y = np.empty(64)
    for i in range(32):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        y[ia] = x[ia] * cos[i] - x[ib] * sin[i]
        y[ib] = x[ib] * cos[i] + x[ia] * sin[i]
    return y


def append_values(kv, positions, table, weight, eps, interleaved) -> np.ndarray:
    """The unrounded rows [T, 576]; rows whose position is out of range are NaN."""
    x, tab = to64(kv), to64(table)
    out = np.full(x.shape, np.nan)
    for t in range(x.shape[0]):
        p = int(positions[t])
        if not 0 <= p < tab.shape[0]:
            continue
        c = x[t, :512]
        if weight is not None:
            c = c / np.sqrt(np.mean(c * c) + eps) * to64(weight)
        out[t, :512] = c
        out[t, 512:] = rotate(x[t, 512:], tab[p, :32], tab[p, 32:], interleaved)
    return out


def fp8_row_values(rows: torch.Tensor) -> np.ndarray:
    """What 656-byte rows stand for, [n, 576] in fp64."""
    rows = rows.cpu()
    n = rows.shape[0]
    code = rows[:, :512].contiguous().view(torch.float8_e4m3fn).float().double().numpy().reshape(n, 4, 128)
    scale = rows[:, 512:528].contiguous().view(torch.float32).double().numpy()
    rope = rows[:, 528:].contiguous().view(torch.bfloat16).double().numpy()
    return np.concatenate([(code * scale[:, :, None]).reshape(n, 512), rope], axis=1)


def q_up(q, w, positions, table, interleaved) -> np.ndarray:
    x, ww, tab = to64(q), to64(w), to64(table)
    T, h, d = x.shape
    out = np.zeros((T, h, 576))
    out[:, :, :512] = np.einsum("thd,hdn->thn", x[:, :, :d - 64], ww)
    for t in range(T):
        p = int(positions[t])
        if 0 <= p < tab.shape[0]:
            for k in range(h):
                out[t, k, 512:] = rotate(x[t, k, d - 64:], tab[p, :32], tab[p, 32:], interleaved)
    return out


def prefix(q, row_values: np.ndarray, pages, prefix_len: int, scale: float):
    """q [T, h, 576], row_values [num_slots, 576] in fp64, pages a list of block numbers; keys of pages
    outside the cache (and rows outside it) take no part.  Returns out [T, h, 512], lse [T, h]."""
    x = to64(q)
    T, h, _ = x.shape
    slots = [int(pages[i // 64]) * 64 + i % 64 for i in range(prefix_len)]
    slots = [s for i, s in enumerate(slots) if int(pages[i // 64]) >= 0 and s < row_values.shape[0]]
    if not slots:
        return np.zeros((T, h, 512)), np.full((T, h), -np.inf)
    rows = row_values[slots]
    s = (x @ rows.T) * scale
    m = s.max(axis=2, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(axis=2, keepdims=True)
    return (e / z) @ rows[:, :512], (m + np.log(z))[:, :, 0]
