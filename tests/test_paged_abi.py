"""The paged-cache entry points' host side, on the CPU: refusals before any HIP call, workspace sizes,
the rotary frequencies, and the binding's checks."""
import ctypes
import math
import pathlib
import re

import numpy as np
import pytest
import torch

from speculative_decoding_verification_specdec_amd import (PagedKvCache, SpecdecError, binding,
                                                           specdec_paged_attention,
                                                           specdec_rope_append,
                                                           specdec_rope_frequencies)

FAKE = 0x1000          # aligned, never dereferenced: every call below fails host-side checks
HEADER = pathlib.Path(__file__).resolve().parents[1] / "include" / "specdec.h"


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, dtype=1, num_pages=10, page_size=16, num_kv_heads=2, head_dim=64,
             max_pages=4, page_stride=2048, slot_stride=128, head_stride=64, page_table=FAKE,
             weight=FAKE, position=FAKE)
    a.update(kw)
    return binding._KvCache(*a.values())


BAD_CACHE = [(dict(num_pages=0), -2), (dict(page_size=0), -2), (dict(num_kv_heads=0), -2),
             (dict(max_pages=0), -2), (dict(head_dim=0), -2), (dict(head_dim=60), -2),
             (dict(head_dim=264), -2), (dict(page_size=1 << 30), -2), (dict(max_pages=1 << 27), -2),
             (dict(page_stride=32), -2), (dict(slot_stride=-128), -2), (dict(head_stride=8), -2),
             (dict(page_stride=1 << 60), -2), (dict(dtype=3), -3), (dict(dtype=-1), -3),
             (dict(k=None), -1), (dict(v=None), -1), (dict(page_table=None), -1),
             (dict(k=FAKE + 8), -4), (dict(v=FAKE + 2), -4), (dict(slot_stride=132), -4),
             (dict(page_stride=2052), -4), (dict(page_table=FAKE + 2), -4),
             (dict(weight=FAKE + 1), -4), (dict(position=FAKE + 2), -4)]


def call_rope(lib, c=None, rope=None, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=128, vs=128, B=3, K=4, heads=8, nd=None, kv=FAKE,
             fp=None, qo=FAKE)
    a.update(kw)
    c = cache() if c is None else c
    rope = binding._Rope(FAKE, 64, 0, 1.0) if rope is None else rope
    return lib.specdec_rope_append(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["B"], a["K"],
                                   a["heads"], a["nd"], a["kv"], a["fp"],
                                   ctypes.byref(rope) if rope else None,
                                   ctypes.byref(c) if c else None, a["qo"], None)


def call_attend(lib, c=None, **kw):
    a = dict(q=FAKE, qs=512, B=3, K=4, heads=8, nd=None, kv=FAKE, scale=0.125, out=FAKE, lse=None,
             ws=FAKE, wsb=1 << 40)
    a.update(kw)
    c = cache() if c is None else c
    return lib.specdec_paged_attention(a["q"], a["qs"], a["B"], a["K"], a["heads"], a["nd"], a["kv"],
                                       a["scale"], ctypes.byref(c) if c else None, a["out"], a["lse"],
                                       a["ws"], a["wsb"], None)


def call_weights(lib, c=None, **kw):
    a = dict(q=FAKE, qs=512, lse=FAKE, B=3, K=4, heads=8, nd=None, acc=None, kv=FAKE, scale=0.125)
    a.update(kw)
    c = cache() if c is None else c
    return lib.specdec_kv_weights(a["q"], a["qs"], a["lse"], a["B"], a["K"], a["heads"], a["nd"],
                                  a["acc"], a["kv"], a["scale"], ctypes.byref(c) if c else None, None)


def call_evict(lib, c=None, **kw):
    a = dict(kv=FAKE, B=3, budget=20, first=2, last=4, new=None, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    c = cache() if c is None else c
    return lib.specdec_kv_evict(ctypes.byref(c) if c else None, a["kv"], a["B"], a["budget"],
                                a["first"], a["last"], a["new"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
@pytest.mark.parametrize("call", [call_rope, call_attend, call_weights, call_evict])
def test_bad_caches_are_refused(lib, call, kw, status):
    assert call(lib, cache(**kw)) == status


@pytest.mark.parametrize("call", [call_rope, call_attend, call_weights, call_evict])
def test_null_cache_and_empty_batch(lib, call):
    assert call(lib, False) == -1
    assert call(lib, B=0, kv=None) == 0
    assert call(lib, B=-1) == -2


@pytest.mark.parametrize("kw,status", [
    (dict(K=-1), -2), (dict(heads=0), -2), (dict(qs=256), -2), (dict(ks=64), -2), (dict(vs=-1), -2),
    (dict(B=1 << 20, K=1 << 12), -2), (dict(qs=1 << 60), -2),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(kv=None), -1),
    (dict(qo=None), -1), (dict(q=FAKE + 8), -4), (dict(qs=516), -4), (dict(ks=132), -4),
    (dict(vs=130), -4), (dict(qo=FAKE + 4), -4), (dict(nd=FAKE + 2), -4), (dict(fp=FAKE + 1), -4),
])
def test_rope_refusals(lib, kw, status):
    assert call_rope(lib, **kw) == status


@pytest.mark.parametrize("rope,status", [
    ((FAKE, 63, 0, 1.0), -2), ((FAKE, -2, 0, 1.0), -2), ((FAKE, 66, 0, 1.0), -2),
    ((FAKE, 64, 0, math.nan), -2), ((FAKE, 64, 0, math.inf), -2), ((None, 64, 0, 1.0), -1),
    ((FAKE + 4, 64, 0, 1.0), -4),
])
def test_rope_parameter_refusals(lib, rope, status):
    assert call_rope(lib, rope=binding._Rope(*rope)) == status
    assert call_rope(lib, rope=False) == -1


@pytest.mark.parametrize("kw,status", [
    (dict(K=-1), -2), (dict(K=64), -2), (dict(heads=7), -2), (dict(heads=0), -2),
    (dict(scale=0.0), -2), (dict(scale=-1.0), -2), (dict(scale=math.nan), -2),
    (dict(scale=math.inf), -2), (dict(qs=100), -2), (dict(q=None), -1), (dict(kv=None), -1),
    (dict(out=None), -1), (dict(ws=None), -1), (dict(q=FAKE + 2), -4), (dict(qs=514), -4),
    (dict(out=FAKE + 8), -4), (dict(lse=FAKE + 2), -4), (dict(ws=FAKE + 8), -4),
    (dict(kv=FAKE + 1), -4), (dict(nd=FAKE + 2), -4), (dict(wsb=8), -5),
])
def test_attention_refusals(lib, kw, status):
    assert call_attend(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=64), -2), (dict(heads=5), -2), (dict(scale=0.0), -2), (dict(q=None), -1),
    (dict(lse=None), -1), (dict(kv=None), -1), (dict(q=FAKE + 2), -4), (dict(lse=FAKE + 2), -4),
    (dict(acc=FAKE + 2), -4), (dict(c=cache(weight=None)), -1),
])
def test_weights_refusals(lib, kw, status):
    assert call_weights(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(budget=0), -2), (dict(first=-1), -2), (dict(last=-1), -2), (dict(first=10, last=11), -2),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), -2), (dict(kv=None), -1), (dict(ws=None), -1),
    (dict(c=cache(weight=None)), -1), (dict(c=cache(position=None)), -1), (dict(ws=FAKE + 4), -4),
    (dict(new=FAKE + 2), -4), (dict(wsb=8), -5),
])
def test_evict_refusals(lib, kw, status):
    assert call_evict(lib, **kw) == status


def test_struct_layouts_follow_the_header():
    src = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    for name, struct in (("specdec_kv_cache", binding._KvCache), ("specdec_rope", binding._Rope)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", src).group(1)
        fields = [re.split(r"[\s*]+", x.strip())[-1] for x in body.split(";") if x.strip()]
        assert fields == [f[0] for f in struct._fields_]
    assert ctypes.sizeof(binding._KvCache) == 88 and ctypes.sizeof(binding._Rope) == 24


def test_workspace_sizes(lib):
    size = lib.specdec_paged_attention_workspace_size
    assert size(0, 5, 32, 8, 128) == 0 and size(4, 64, 32, 8, 128) == 0
    assert size(4, 5, 30, 8, 128) == 0 and size(4, 5, 32, 8, 12) == 0
    assert size(4, 5, 32, 8, 128) >= 16 and size(4, 5, 32, 8, 128) % 16 == 0
    c = cache()
    ev = lib.specdec_kv_evict_workspace_size
    assert ev(0, ctypes.byref(c), 20) == 0 and ev(3, ctypes.byref(c), 0) == 0
    assert ev(3, ctypes.byref(c), 20) >= 16


def test_rope_frequencies_by_their_formulas():
    f = specdec_rope_frequencies(8, 10000.0)
    assert np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    assert np.allclose(specdec_rope_frequencies(8, 10000.0, scaling="linear", factor=4.0), f / 4,
                       rtol=1e-14)
    g = specdec_rope_frequencies(8, 10000.0, scaling="base", factor=4.0)
    assert g[0] == 1.0 and np.allclose(g[-1], f[-1] / 4, rtol=1e-12)   # the slowest pair, exactly
    # Turns over 1000 positions: 159, 15.9, 1.59, 0.159; kept from 32, divided up to 1, blended between.
    t = specdec_rope_frequencies(8, 10000.0, scaling="turns", factor=4.0, original_len=1000.0)
    w = (1000 * f / (2 * math.pi) - 1) / 31
    w = np.clip(w, 0, 1)
    assert np.allclose(t, w * f + (1 - w) * f / 4, rtol=1e-13)
    assert t[0] == f[0] and t[3] == f[3] / 4


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=258), dict(base=1.0), dict(base=math.nan),
    dict(base=math.inf), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.nan),
    dict(rotary_dim=2, scaling="base", factor=2.0), dict(scaling="turns", factor=2.0),
    dict(scaling="turns", factor=2.0, original_len=10.0, turns_low=3.0, turns_high=3.0),
    dict(scaling="other"),
])
def test_rope_frequency_refusals(kw):
    with pytest.raises(SpecdecError):
        specdec_rope_frequencies(kw.pop("rotary_dim", 8), kw.pop("base", 10000.0), **kw)


def pools(dtype=torch.bfloat16, shape=(6, 4, 2, 16)):
    return torch.zeros(shape, dtype=dtype), torch.zeros(shape, dtype=dtype)


def test_binding_checks_the_cache():
    k, v = pools()
    table = torch.zeros(2, 3, dtype=torch.int32)
    PagedKvCache(k, v, table)
    PagedKvCache(k.transpose(1, 2), v.transpose(1, 2), table)
    for bad in (lambda: PagedKvCache(k[0], v[0], table), lambda: PagedKvCache(k, v[:3], table),
                lambda: PagedKvCache(k, v.float(), table),
                lambda: PagedKvCache(k.long(), v.long(), table),
                lambda: PagedKvCache(k, v.transpose(1, 2).contiguous().transpose(1, 2), table),
                lambda: PagedKvCache(k.transpose(2, 3), v.transpose(2, 3), table),
                lambda: PagedKvCache(k, v, table.long()), lambda: PagedKvCache(k, v, table[0]),
                lambda: PagedKvCache(k, v, table, weight=torch.zeros(6, 4, 2)),
                lambda: PagedKvCache(k, v, table, position=torch.zeros(6, 2, 4))):
        with pytest.raises(SpecdecError):
            bad()


def test_binding_checks_the_round():
    k, v = pools()
    c = PagedKvCache(k, v, torch.zeros(2, 3, dtype=torch.int32))
    kv = torch.zeros(2, dtype=torch.int32)
    q, kn = torch.zeros(2, 3, 4, 16, dtype=k.dtype), torch.zeros(2, 3, 2, 16, dtype=k.dtype)
    for bad in (lambda: specdec_paged_attention(q, c, kv),                       # a CPU cache
                lambda: specdec_paged_attention(q[0], c, kv),
                lambda: specdec_paged_attention(q.float(), c, kv),
                lambda: specdec_paged_attention(q[:1], c, kv),
                lambda: specdec_paged_attention(q[..., :8], c, kv),
                lambda: specdec_paged_attention(q, c, kv.long()),
                lambda: specdec_paged_attention(q, c, kv, num_draft=kv[:1]),
                lambda: specdec_paged_attention(q.transpose(1, 2), c, kv),
                lambda: specdec_rope_append(q, kn, kn[:, :2], c, kv, None),
                lambda: specdec_rope_append(q, kn[..., :8], kn, c, kv, None),
                lambda: specdec_rope_append(q, kn, kn, c, kv, torch.zeros(4)),
                lambda: specdec_rope_append(q, kn, kn, c, kv, None, out=q.float())):
        with pytest.raises(SpecdecError):
            bad()


@pytest.mark.parametrize("call", [call_rope, call_attend, call_weights, call_evict])
def test_limits_of_a_cache(lib, call):
    # 2^30 slots a sequence and 65536 kv heads; one more of either would pass 32 bits in a kernel.
    # (An empty batch: nothing is launched.)
    most = dict(page_size=1 << 20, max_pages=1 << 10, slot_stride=64, page_stride=64 << 20, num_kv_heads=1)
    assert call(lib, cache(**most), B=0, heads=1) == 0 if call is not call_evict else call(lib, cache(**most), B=0) == 0
    assert call(lib, cache(**{**most, "max_pages": (1 << 10) + 1}), B=0, kv=FAKE) == -2
    assert call(lib, cache(num_kv_heads=65537, slot_stride=64 * 65537, page_stride=1024 * 65537)) == -2


def test_rope_in_place_wants_a_dense_q(lib):
    # q_out = q with tokens further apart than their rows: a token's output would lie in another's input.
    assert call_rope(lib, q=2 * FAKE, qo=2 * FAKE, qs=1024) == -2
    assert call_rope(lib, q=2 * FAKE, qo=2 * FAKE, qs=1024, heads=2 ** 31 - 1, B=1, K=0) == -2


def test_evict_wants_new_len_apart_from_kv_len_or_in_its_place(lib):
    for off in (-8, -4, 4, 8):
        assert call_evict(lib, kv=2 * FAKE, new=2 * FAKE + off) == -2
    for off in (0, -12, 12):            # (told apart by the next check)
        assert call_evict(lib, kv=2 * FAKE, new=2 * FAKE + off, wsb=8) == -5
