"""The life of a drafting batch (tests/test_gpu_drafted.py) held to the tolerance of the attention
alone: the rotated keys in the cache and the rotated queries are checked for themselves, and
the replay then attends over what is stored, with masks, positions and lengths of its own.

Rotated elements: tests/test_gpu_rotary_axes.py (amplitude 1).  Outputs: tests/test_gpu_tree.py.  A
token more or less of 33 moves an output of random values by about 0.03; the tolerance there is below
0.01 in bf16.
"""
import numpy as np
import pytest
import torch

import test_gpu_drafted as life
import test_gpu_tree as tree
from helpers import dev, f64
from paged_kv_decode_10_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


class Exact(life.Replay):
    queries = []          # rotated ones of every layer of the last call, as the kernels got them
    checked = 0

    def near(self, got, x, pos):
        """``got``: x rotated at ``pos``, in storage precision."""
        want = self.rotated(x, pos)
        n = self.dec.d // 2
        size = np.abs(x[..., :n]) + np.abs(x[..., n:])
        tol = np.concatenate([size, size], -1) * 2.0**-21 + tree.U[self.dec.dtype] * np.abs(want)
        assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()

    def check(self, out, sid, first, q, pos, sees):
        dec, row = self.dec, self.rows[sid]
        n, total = q.shape[1], self.held(sid)
        assert len(self.queries) == dec.n_layers and dec.alloc.seq_len(sid) == total
        blocks = torch.tensor(dec.alloc.seq_blocks(sid), device=dev())
        for layer in range(dec.n_layers):
            k, v, p = (np.concatenate([x[layer] for x in row["k"]]), np.concatenate([x[layer] for x in row["v"]]),
                       np.concatenate(row["p"], axis=1))
            stored = [f64(c[layer][blocks]).transpose(0, 2, 1, 3).reshape(-1, dec.Hkv, dec.d)[:total]
                      for c in (dec.k_caches, dec.v_caches)]
            self.near(stored[0], k, p)
            assert np.array_equal(stored[1], v)
            qr = f64(self.queries[layer])[first:first + n]
            self.near(qr, q[layer], pos)
            for h in range(dec.Hq):
                ks, vs = (x[:, h // (dec.Hq // dec.Hkv)] for x in stored)
                s = np.where(sees, qr[:, h] @ ks.T * dec.scale, -np.inf)
                m = s.max(1, keepdims=True)
                w = np.exp(s - m)
                lse = m[:, 0] + np.log(w.sum(1))
                w /= w.sum(1, keepdims=True)
                swing = dec.scale * np.where(sees, np.abs(qr[:, h]) @ np.abs(ks).T, 0).max(1)
                tree.check(out[layer, first:first + n, h], None, (w @ vs, lse, w @ np.abs(vs), swing), dec.dtype,
                           dec.d)
        Exact.checked += n


@pytest.mark.parametrize("dtype,L,sections", [("f32", 2, None), ("bf16", 1, (8, 12, 12)), ("bf16", 3, None),
                                              ("f32", 1, (8, 12, 12)), ("f32", 3, None), ("bf16", 2, (20, 12))])
def test_life_of_a_drafting_batch_to_the_last_bit_that_counts(dtype, L, sections, monkeypatch):
    real, call = binding.decode_attn_tree_args, life.DraftDecoder._run

    def noted(args, stream=None):
        Exact.queries.append(args.keep[0].clone())
        real(args, stream)

    def fresh(self, *args):
        Exact.queries.clear()
        return call(self, *args)
    monkeypatch.setattr(binding, "decode_attn_tree_args", noted)
    monkeypatch.setattr(life.DraftDecoder, "_run", fresh)
    monkeypatch.setattr(life, "Replay", Exact)
    Exact.checked = 0
    life.test_life_of_a_drafting_batch(dtype, L, sections)
    assert Exact.checked > 200
