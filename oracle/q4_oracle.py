"""fp64 reference of the 4-bit weight format (include/moe.h): a matrix [rows, cols] is
W[r, c] = s[c // G, r] * (q[r, c] - 8), codes q in 0..15, one bf16 scale per group of G columns."""
from __future__ import annotations

import numpy as np
import torch

# column of an 8-column block that nibble i of its 32-bit word holds
NIBBLE_COLUMN = (0, 2, 4, 6, 1, 3, 5, 7)


def pack(q: np.ndarray) -> np.ndarray:
    """Codes [.., rows, cols] in 0..15 -> bytes [.., rows, cols / 2]."""
    blocks = q.astype(np.uint32).reshape(*q.shape[:-1], -1, 8)
    word = np.zeros(blocks.shape[:-1], dtype=np.uint32)
    for i, c in enumerate(NIBBLE_COLUMN):
        word |= blocks[..., c] << np.uint32(4 * i)
    return word.astype("<u4").view(np.uint8).reshape(*q.shape[:-1], -1)


def unpack(codes: np.ndarray) -> np.ndarray:
    """The inverse of pack."""
    word = np.ascontiguousarray(codes).view("<u4")
    q = np.empty((*word.shape, 8), dtype=np.int64)
    for i, c in enumerate(NIBBLE_COLUMN):
        q[..., c] = (word >> np.uint32(4 * i)) & 15
    return q.reshape(*codes.shape[:-1], -1)


def quantize(W: torch.Tensor, group: int):
    """W bf16 [mats, rows, cols] -> codes uint8 [mats, rows, cols/2], scales bf16 [mats, cols/group, rows to 8]."""
    mats, rows, cols = W.shape
    w = W.double().numpy().reshape(mats, rows, cols // group, group)
    with np.errstate(invalid="ignore"):
        top = np.abs(w).max(-1)
        s = torch.from_numpy(top / 7).to(torch.bfloat16)
        sf = s.double().numpy()[..., None]
        ok = np.isfinite(sf) & (sf > 0)
        q = np.where(ok, np.clip(np.rint(w / np.where(ok, sf, 1.0)), -8, 7), 0.0)
    codes = pack(np.nan_to_num(q).astype(np.int64).reshape(mats, rows, cols) + 8)
    scales = torch.zeros(mats, cols // group, -(-rows // 8) * 8, dtype=torch.bfloat16)
    scales[:, :, :rows] = s.transpose(1, 2)
    return torch.from_numpy(codes), scales


def values(codes: torch.Tensor, scales: torch.Tensor, group: int) -> np.ndarray:
    """fp64 values [mats, rows, cols] of codes and scales."""
    q = unpack(codes.cpu().numpy()) - 8
    mats, rows, cols = q.shape
    s = scales.double().cpu().numpy()[:, :, :rows].transpose(0, 2, 1)[..., None]
    with np.errstate(invalid="ignore"):
        return (q.reshape(mats, rows, cols // group, group) * s).reshape(mats, rows, cols)
