"""Pins of the paged-cache oracle (CPU): library routines, hand-worked cases and invariants."""
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from paged_cases import make_round, wide


def test_rope_row_turns_pairs_and_keeps_scores_of_equal_distance():
    f = np.array([1.0, 0.25])
    x = np.array([1.0, 2.0, 3.0, 4.0, 9.0])
    y = po.rope_row(x, 2, f, False, 1.0)
    want = [math.cos(2) - 3 * math.sin(2), 2 * math.cos(.5) - 4 * math.sin(.5),
            3 * math.cos(2) + math.sin(2), 4 * math.cos(.5) + 2 * math.sin(.5), 9.0]
    assert np.allclose(y, want, rtol=1e-15)
    z = po.rope_row(x, 2, f, True, 1.0)
    assert np.allclose(z[:2], [math.cos(2) - 2 * math.sin(2), 2 * math.cos(2) + math.sin(2)])
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal(4), rng.standard_normal(4)
    for inter in (False, True):     # scores depend on the distance alone
        s = [po.rope_row(q, 7 + o, f, inter, 1.0) @ po.rope_row(k, 3 + o, f, inter, 1.0)
             for o in (0, 1000, 123456)]
        assert np.allclose(s, s[0], atol=1e-9)


@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (6, 2)])
def test_attention_is_torchs_softmax_of_masked_scores(heads, kv_heads):
    r = make_round([5, 0, 17], 2, heads, kv_heads, 16, 4, "f32", seed=1)
    out, lse, _, _ = po.paged_attention(wide(r.q), wide(r.k), wide(r.v), wide(r.table), wide(r.kv_len),
                                        scale=r.scale)
    for b, L in enumerate((5, 0, 17)):
        slots = torch.arange(L + 3)
        ids = r.table[b].long()[slots // 4]
        k = r.k[ids, slots % 4].double().repeat_interleave(heads // kv_heads, 1)
        v = r.v[ids, slots % 4].double().repeat_interleave(heads // kv_heads, 1)
        x = torch.einsum("ihd,jhd->hij", r.q[b].double(), k) * r.scale
        x = x.masked_fill(slots[None, None] > L + torch.arange(3)[None, :, None], -math.inf)
        want = torch.einsum("hij,jhd->ihd", x.softmax(-1), v)
        assert np.allclose(out[b], want.numpy(), rtol=1e-12, atol=1e-14)
        assert np.allclose(lse[b], x.logsumexp(-1).t().numpy(), rtol=1e-12)


def test_invalid_sequences_are_nan_and_padding_zero():
    r = make_round([3, 3, 3, 3], 2, 2, 1, 8, 4, "f32", seed=2)
    nd = np.array([1, 3, 2, 2])
    kv = np.array([3, 3, -1, 3])
    table = wide(r.table)
    table[3, 0] = 10 ** 6
    out, lse, _, _ = po.paged_attention(wide(r.q), wide(r.k), wide(r.v), table, kv, num_draft=nd)
    assert np.isfinite(out[0, :2]).all() and (out[0, 2] == 0).all() and (lse[0, 2] == -np.inf).all()
    assert np.isnan(out[1:]).all() and np.isnan(lse[1:]).all()


def test_weights_of_all_rows_sum_to_the_number_of_rows():
    r = make_round([6, 1, 11], 3, 6, 2, 8, 4, "f32", seed=3)
    a = [wide(x) for x in (r.q, r.k, r.v, r.table, r.kv_len)]
    _, lse, _, _ = po.paged_attention(*a, scale=r.scale)
    w0 = np.zeros(wide(r.weight).shape)
    w, added, _ = po.kv_weights(a[0], lse, a[1], a[3], a[4], w0, scale=r.scale)
    assert np.allclose(w.sum(), 3 * 4 * 6) and np.allclose(w, added)
    # Only the accepted rows count, and rejected slots are left alone.
    w1, _, _ = po.kv_weights(a[0], lse, a[1], a[3], a[4], w0, scale=r.scale,
                             accept_len=np.array([0, -1, 3]))
    assert np.allclose(w1.sum(), (1 + 0 + 4) * 6)


def test_evict_by_hand():
    # Six slots, one head, budget 3: the first position and the newest are protected, of the others
    # the heaviest (slot 4) stays; movers 4, 5 fill the holes 1, 2.
    k = np.arange(8.0).reshape(2, 4, 1, 1)
    w = np.array([[[.1, .5, .4, .3]], [[.6, .2, 0, 0]]])
    p = np.array([[[0, 1, 2, 3]], [[4, 5, 0, 0]]])
    table = np.array([[0, 1]])
    nk, nv, nw, npos, n = po.kv_evict(k, -k, table, [6], w, p, 3, keep_first=1, keep_last=1)
    assert n.tolist() == [3]
    assert nk.reshape(-1)[:3].tolist() == [0, 4, 5] and (nv == -nk).all()
    assert npos.reshape(-1)[:3].tolist() == [0, 4, 5] and nw.reshape(-1)[:3].tolist() == [.1, .6, .2]
    assert nk.reshape(-1)[3:].tolist() == [3, 4, 5, 6, 7]
    # Ties keep the lower slot, NaN goes first, a short sequence stays, a bad length is reported.
    w[:] = 1.0
    w[0, 0, 0] = np.nan
    nk, _, _, _, n = po.kv_evict(k, -k, table, [6], w, p, 3)
    assert nk.reshape(-1)[:3].tolist() == [3, 1, 2]
    assert po.kv_evict(k, -k, table, [3], w, p, 3)[4].tolist() == [3]
    assert po.kv_evict(k, -k, table, [9], w, p, 3)[4].tolist() == [-1]
