"""Block keys, block scores and attention over listed blocks in fp64 -- TEST INFRASTRUCTURE ONLY.

Plain definitions over a stream's contiguous rows (float64 [len][512] latent and [len][64] rope).
Pooled keys and weighted sums of rectified products are the pages' way to choose rows (issue #1142,
"What happens now" and piece 2); the chosen rows are attended as issue #1313, step 2 describes.
"""
from __future__ import annotations

import numpy as np

BLOCK = 64


def blocks_of(n: int) -> int:
    return -(-n // BLOCK)


def block_keys(lat: np.ndarray, rope: np.ndarray) -> np.ndarray:
    """The mean row of each block: float64 [blocks][576]."""
    rows = np.concatenate([np.asarray(lat, np.float64), np.asarray(rope, np.float64)], axis=1)
    return np.stack([rows[a:a + BLOCK].sum(0) / len(rows[a:a + BLOCK]) for a in range(0, len(rows), BLOCK)])


def block_scores(q: np.ndarray, keys: np.ndarray, length: int, w, scale: float, sink: int, local: int) -> np.ndarray:
    """q: [R][H][576]; keys: [blocks][576]; w: [R][H] or None.  float64 [R][blocks]: +inf for forced blocks,
    -inf for those behind the row's own."""
    R = q.shape[0]
    out = np.full((R, blocks_of(length)), -np.inf)
    for r in range(R):
        own = (length - R + r) // BLOCK
        for b in range(own + 1):
            if b < sink or b > own - local:
                out[r, b] = np.inf
                continue
            d = np.maximum(scale * (q[r].astype(np.float64) @ keys[b]), 0.0)
            out[r, b] = d.sum() if w is None else float(np.dot(np.asarray(w[r], np.float64), d))
    return out


def rows_of_list(blocks, pos: int) -> np.ndarray:
    """The rows that a query at `pos` sees of its listed blocks, in list order."""
    got = [np.arange(b * BLOCK, min(b * BLOCK + BLOCK, pos + 1)) for b in blocks if b >= 0]
    return np.concatenate(got) if got else np.zeros(0, np.int64)


def attend_rows(q: np.ndarray, lat: np.ndarray, rope: np.ndarray, rows, scale: float):
    """Attention of one query row's heads ([H][576]) over the given rows: (out [H][512], lse [H]); zero and
    -inf where there is no row."""
    H = q.shape[0]
    if len(rows) == 0:
        return np.zeros((H, 512)), np.full(H, -np.inf)
    c, k = np.asarray(lat, np.float64)[rows], np.asarray(rope, np.float64)[rows]
    s = scale * (q[:, :512].astype(np.float64) @ c.T + q[:, 512:].astype(np.float64) @ k.T)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    return e @ c / e.sum(1, keepdims=True), (m + np.log(e.sum(1, keepdims=True)))[:, 0]
