"""Cases of tree verification and cross attention: inputs from a seed, float64
references and derived error bounds."""
from __future__ import annotations

import numpy as np
import torch

import paged_kv_cache_122_gb300 as pk
from oracle import tree_ref as R

DEV = "cuda:0"


def bits(t: torch.Tensor) -> np.ndarray:
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype).to(DEV)


def parents_of(n: int, rng) -> list:
    return [-1] + [int(rng.integers(max(0, r - 6), r)) for r in range(1, n)]


class Case:
    """Sequences of ``lens`` keys with ``rows`` query rows each over a shuffled pool."""

    def __init__(self, seed, lens, rows, G, Hkv, D, B, tree, words=None, strength=2.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.rows, self.B, self.D, self.Hkv, self.H = list(lens), list(rows), B, D, Hkv, G * Hkv
        need = [-(-n // B) for n in lens]
        self.blocks = sum(need) + 5
        ids = rng.permutation(self.blocks).astype(np.int32)
        self.tables = np.full((len(lens), max(1, max(need, default=1)) + 1), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        T = int(self.cu[-1])

        def bf16(*shape, gain=1.0):
            return (gain * torch.randn(*shape, generator=gen)).to(torch.bfloat16)
        self.q = bf16(T, self.H, D, gain=strength).to(DEV)
        self.k = bf16(self.blocks, B, Hkv, D).to(DEV)
        self.v = bf16(self.blocks, B, Hkv, D).to(DEV)
        self.scale = D ** -0.5
        self.mask = None
        if tree:
            words = words or max(1, -(-max(rows, default=1) // 64))
            self.parents = [parents_of(n, rng) if n else [] for n in rows]
            self.mask = np.concatenate([R.ancestors_mask(p, words) for p in self.parents] or
                                       [np.zeros((0, words), np.uint64)])
        self.rng = rng

    def run(self, out_dtype=torch.float32, **kw):
        args = dict(out_dtype=out_dtype, max_seq_len=max(self.lens, default=0))
        args.update(kw)
        common = (self.k, self.v, dev(self.tables), dev(np.asarray(self.lens, np.int32)), self.scale)
        cu, most = dev(self.cu), max(self.rows, default=0)
        if self.mask is not None:
            return pk.paged_attention_tree(self.q, cu, most, dev(self.mask.view(np.int64)), *common, **args)
        return pk.paged_attention_cross(self.q, cu, most, *common, **args)

    def reference(self):
        return R.masked_attention(bits(self.q), bits(self.k), bits(self.v), self.tables, self.lens, self.cu, self.scale,
                                  self.B, self.mask)

    def check(self, out, what="", rows=None):
        ref, spread, size, most = self.reference()
        tol = R.bound(ref, spread, size, most, max(self.lens), self.D, out.dtype == torch.bfloat16)
        got = out.double().cpu().numpy()
        rows = slice(None) if rows is None else rows
        err = np.abs(got - ref)[rows]
        assert np.all(np.isfinite(got[rows])), f"{what}: non-finite output"
        worst = np.unravel_index(np.argmax(err / tol[rows]), err.shape)
        assert np.all(err <= tol[rows]), f"{what}: off by {err[worst]:.3e} at {worst}, allowed {tol[rows][worst]:.3e}"
        return float((err / tol[rows]).max())


def clean():
    assert pk.pk_get_device_error() == 0
