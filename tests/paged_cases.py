"""Seeded paged caches and rounds for the tests of the paged-cache entry points: scattered pages,
table entries past the used slots that are no page ids, pools whose unused slots hold NaN."""
from dataclasses import dataclass

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# Half a step of each type relative to the value (for float32 too).
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@dataclass
class Round:
    dtype: str
    q: torch.Tensor          # [B, T, H, D] on the CPU, in dtype
    k: torch.Tensor          # pools [P, page, Hkv, D]
    v: torch.Tensor
    k_new: torch.Tensor      # [B, T, Hkv, D]
    v_new: torch.Tensor
    table: torch.Tensor      # [B, max_pages] int32
    kv_len: torch.Tensor     # [B] int32
    num_draft: torch.Tensor | None
    weight: torch.Tensor     # [P, Hkv, page] float32
    position: torch.Tensor   # [P, Hkv, page] int32
    scale: float

    @property
    def K(self):
        return self.q.shape[1] - 1


def wide(t):
    """A tensor as a numpy array the oracle takes: float64, or integers."""
    return t.double().numpy() if t.is_floating_point() else t.numpy().astype(np.int64)


def make_round(lens, K, heads, kv_heads, dim, page, dtype, *, seed, ragged=False, spare=2,
               q_scale=1.5, used_extra=0):
    """Sequences of ``lens`` slots before a round of K + 1 tokens.  ``used_extra`` more slots a sequence
    get pages.  The round's own slots (kv_len .. kv_len + K) are filled as if appended."""
    g = torch.Generator().manual_seed(seed)
    B, T = len(lens), K + 1
    d = DTYPES[dtype]
    max_pages = -(-(max(lens) + T + used_extra) // page) + 1
    need = [-(-(L + T + used_extra) // page) for L in lens]
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, max_pages), -7, dtype=torch.int32)
    table[:, 1::2] = 2 ** 31 - 1            # entries past the used slots are no page ids
    k = torch.full((pages, page, kv_heads, dim), float("nan"), dtype=d)
    v = k.clone()
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
        for j in range(lens[b] + T):
            p, o = int(table[b, j // page]), j % page
            k[p, o] = torch.randn(kv_heads, dim, generator=g).to(d)
            v[p, o] = torch.randn(kv_heads, dim, generator=g).to(d)
    nd = torch.randint(0, K + 1, (B,), generator=g, dtype=torch.int32) if ragged else None
    return Round(dtype, (torch.randn(B, T, heads, dim, generator=g) * q_scale).to(d), k, v,
                 torch.randn(B, T, kv_heads, dim, generator=g).to(d),
                 torch.randn(B, T, kv_heads, dim, generator=g).to(d), table,
                 torch.tensor(lens, dtype=torch.int32), nd,
                 torch.rand(pages, kv_heads, page, generator=g),
                 torch.randint(0, 10 ** 6, (pages, kv_heads, page), generator=g, dtype=torch.int32),
                 dim ** -0.5)
