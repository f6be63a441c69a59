"""The cache operators without a GPU: the calls refuse bad arguments on the host
before anything is launched, and their oracle agrees with the causal oracle and
with examples worked out by hand."""
import ctypes
import os
import re

import numpy as np
import pytest

from llama_decoder_only_rmsnorm_b200 import binding as B
from oracle import cache_oracle as C
from oracle import llama3_oracle as O

FAKE = 1 << 20   # an aligned, never-dereferenced address: these calls must fail first
ARG, ALIGN, WORKSPACE = 1, 2, 3


def cfg(**kw):
    d = dict(dim=4096, n_heads=32, n_kv_heads=8, ffn_hidden=14336, vocab=128256)
    d.update(kw)
    return B.make_config(**d)


def test_tree_attention_refuses_bad_arguments():
    c, lib = cfg(), B.lib()
    need = B.llama3_tree_workspace_size(c, 2, 16, 64)

    def call(conf=c, q=FAKE, kc=FAKE, lens=FAKE, kn=FAKE, par=FAKE, out=FAKE, cap=64, max_len=64, batch=2, nodes=16,
             ws=FAKE, ws_bytes=1 << 40):
        return lib.llama3_attention_tree(ctypes.byref(conf), q, kc, FAKE, cap, lens, max_len, kn, FAKE, par, batch,
                                         nodes, out, ws, ws_bytes, None)
    assert call(conf=cfg(dim=4000)) == ARG
    for name in ("q", "kc", "lens", "kn", "par", "out"):
        assert call(**{name: None}) == ARG, name
        assert call(**{name: FAKE + 2}) == ALIGN, name
    assert call(q=FAKE + 8) == ALIGN
    assert call(nodes=0) == ARG
    assert call(nodes=257) == ARG
    assert call(batch=0) == ARG
    assert call(max_len=65) == ARG
    assert call(max_len=-1) == ARG
    assert call(cap=0, max_len=0) == ARG
    if need:
        assert call(ws=None) == WORKSPACE
        assert call(ws_bytes=need - 1) == WORKSPACE
        assert call(ws=FAKE + 8) == ALIGN
    for bad in (dict(batch=0), dict(n_nodes=257), dict(max_len=-1)):
        args = dict(batch=2, n_nodes=16, max_len=64, **{}) | bad
        with pytest.raises(B.Llama3Error) as e:
            B.llama3_tree_workspace_size(c, **args)
        assert e.value.status == ARG


def test_observed_attention_refuses_bad_arguments():
    c, lib = cfg(), B.lib()
    need = B.llama3_observe_workspace_size(c, 2, 16, 48)

    def call(q=FAKE, kc=FAKE, out=FAKE, cap=64, batch=2, seq=16, lens=FAKE, rows=FAKE, max_len=48, win=FAKE, w=FAKE,
             pos=FAKE, slot_pos=FAKE, ws=FAKE, ws_bytes=1 << 40):
        return lib.llama3_attention_observed(ctypes.byref(c), q, kc, FAKE, cap, batch, seq, lens, rows, max_len, out,
                                             win, w, pos, slot_pos, ws, ws_bytes, None)
    for name in ("q", "kc", "out", "w"):
        assert call(**{name: None}) == ARG, name
    for name in ("q", "kc", "out", "w", "lens", "rows", "win", "pos", "slot_pos"):
        assert call(**{name: FAKE + 2}) == ALIGN, name
    assert call(seq=17) == ARG                 # max_len + seq > cache_cap
    assert call(seq=0) == ARG
    assert call(batch=0) == ARG
    assert call(max_len=-1) == ARG
    assert call(max_len=2 ** 31 - 1) == ARG    # no wrap of the sum
    assert call(ws=None) == WORKSPACE
    assert call(ws_bytes=need - 1) == WORKSPACE
    assert call(ws=FAKE + 8) == ALIGN
    with pytest.raises(B.Llama3Error):
        B.llama3_observe_workspace_size(c, 2, 0, 48)


def _caches(n, **kw):
    d = dict(k=FAKE, v=FAKE, weights=FAKE, slot_pos=FAKE)
    d.update(kw)
    return (B.llama3_bounded_cache * n)(*[B.llama3_bounded_cache(**d) for _ in range(n)])


def test_eviction_refuses_bad_arguments():
    c, lib = cfg(), B.lib()
    need = B.llama3_evict_workspace_size(c, 2, 3, 100, 10)
    other = 1 << 22

    def call(src=_caches(2), src_cap=100, dst=None, dst_cap=0, layers=2, batch=3, lens=FAKE, max_len=100, budget=10,
             recent=4, pos=FAKE, lens_out=FAKE, ws=FAKE, ws_bytes=1 << 40):
        return lib.llama3_cache_evict(ctypes.byref(c), src, src_cap, dst, dst_cap, layers, batch, lens, max_len,
                                      budget, recent, pos, lens_out, ws, ws_bytes, None)
    assert call(src=None) == ARG
    for name in ("k", "v", "weights", "slot_pos"):
        assert call(src=_caches(2, **{name: None})) == ARG, name
        assert call(src=_caches(2, **{name: FAKE + 2})) == ALIGN, name
    full = dict(k=other, v=other, weights=other, slot_pos=other)
    assert call(dst=_caches(2, **full), dst_cap=9) == ARG          # does not hold the budget
    assert call(dst=_caches(2, **dict(full, v=None)), dst_cap=10) == ARG
    assert call(dst=_caches(2, **dict(full, k=FAKE)), dst_cap=10) == ARG   # shares a buffer with the source
    for name in ("lens", "pos", "lens_out"):
        assert call(**{name: None}) == ARG, name
        assert call(**{name: FAKE + 2}) == ALIGN, name
    assert call(layers=0) == ARG
    assert call(batch=0) == ARG
    assert call(max_len=101) == ARG
    assert call(max_len=-1) == ARG
    assert call(budget=0) == ARG
    assert call(recent=-1) == ARG
    assert call(recent=11) == ARG
    assert call(ws=None) == WORKSPACE
    assert call(ws_bytes=need - 1) == WORKSPACE
    assert call(ws=FAKE + 8) == ALIGN
    with pytest.raises(ValueError):
        B.llama3_cache_evict(c, _caches(2), 100, _caches(1, **full), 10, 3, None, 100, 10, 4, None, None, None, 0)


def test_acceptance_refuses_bad_arguments():
    c, lib = cfg(), B.lib()
    names = ("draft", "target", "par", "lens", "path", "acc", "nxt", "lens_out")

    def accept(batch=2, nodes=8, pos=FAKE, pos_out=FAKE, **kw):
        p = [kw.get(n, FAKE) for n in names]
        return lib.llama3_tree_accept(*p[:3], batch, nodes, *p[3:], pos, pos_out, None)
    for name in names:
        assert accept(**{name: None}) == ARG, name
        assert accept(**{name: FAKE + 2}) == ALIGN, name
    assert accept(batch=0) == ARG
    assert accept(nodes=0) == ARG
    assert accept(nodes=257) == ARG
    assert accept(pos=None) == ARG             # positions_out without positions
    assert accept(pos=FAKE + 2) == ALIGN

    def commit(nodes=_caches(2), caches=_caches(2), cap=64, layers=2, batch=2, n=8, path=FAKE, acc=FAKE, lens=FAKE,
               pos=None):
        return lib.llama3_tree_commit(ctypes.byref(c), nodes, caches, cap, layers, batch, n, path, acc, lens, pos,
                                      None)
    assert commit(nodes=None) == ARG
    assert commit(caches=None) == ARG
    assert commit(nodes=_caches(2, k=None)) == ARG
    assert commit(caches=_caches(2, v=None)) == ARG
    assert commit(caches=_caches(2, v=FAKE + 8)) == ALIGN
    assert commit(caches=_caches(2, slot_pos=FAKE + 2)) == ALIGN
    assert commit(cap=0) == ARG
    assert commit(layers=0) == ARG
    assert commit(n=257) == ARG
    for name in ("path", "acc", "lens"):
        assert commit(**{name: None}) == ARG, name
        assert commit(**{name: FAKE + 2}) == ALIGN, name
    with pytest.raises(ValueError):
        B.llama3_tree_commit(c, _caches(2), _caches(1), 64, 2, 8, None, None, None)


def test_what_no_kernel_takes_is_refused():
    unsupported = 7
    wide = B.make_config(65 * 16, 65, 1, 64, dtype="f32")       # more query heads per KV head than a tile has rows
    wide16 = B.make_config(129 * 64, 129, 1, 64)
    for c in (wide, wide16):
        for size in (lambda: B.llama3_tree_workspace_size(c, 1, 4, 10), lambda: B.llama3_observe_workspace_size(c, 1, 4, 10)):
            with pytest.raises(B.Llama3Error) as e:
                size()
            assert e.value.status == unsupported
    with pytest.raises(B.Llama3Error) as e:     # more pieces of work than the plan counts
        B.llama3_observe_workspace_size(cfg(), 8, 1 << 20, 0)
    assert e.value.status == unsupported
    assert B.llama3_tree_workspace_size(B.make_config(128 * 64, 128, 1, 64), 1, 4, 10) > 0
    assert B.llama3_tree_workspace_size(cfg(), 1, 4, 0) == 0    # nothing cached: nothing to keep


def test_tree_oracle_of_a_chain_is_causal_attention():
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((1, n, h, 8)) for n, h in ((5, 4), (12, 2), (12, 2)))
    want = O.gqa_attention(q[0], k[0], v[0], start_pos=7)
    par = np.array([[-1, 0, 1, 2, 3]])
    got, _, _ = C.tree_attention(q, k[:, :7], v[:, :7], [7], k[:, 7:], v[:, 7:], par)
    np.testing.assert_allclose(got[0], want, rtol=1e-12, atol=1e-12)


def test_observed_oracle_weights_sum_to_the_rows():
    rng = np.random.default_rng(4)
    q, k, v = (rng.standard_normal((2, n, h, 8)) for n, h in ((5, 4), (12, 2), (12, 2)))
    out, _, _, w = C.observed_attention(q, k, v, [7, 2], [5, 3], None)
    np.testing.assert_allclose(out[0], O.gqa_attention(q[0], k[0], v[0], start_pos=7), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(w[0].sum(), 5 * 4)          # every row hands out a weight of 1 per head
    np.testing.assert_allclose(w[1, :, :5].sum(), 3 * 4)
    assert np.isnan(w[1, :, 5:]).all() and not out[1, 3:].any()


def test_eviction_oracle_by_hand():
    # positions 0..7 in order, budget 4, the last two kept: 6, 7 and the two largest weights (5.0 at 1, 3.0 at 4)
    w = np.array([1.0, 5.0, 2.0, 0.0, 3.0, 0.5, 0.0, 9.0])
    assert C.evict_sources(w, np.arange(8), 8, 8, 4, 2) == [4, 1, 6, 7]
    # ties go to the lower slot; a NaN is kept before any number
    assert C.evict_sources(np.zeros(6), np.arange(6), 6, 6, 3, 0) == [0, 1, 2]
    assert C.evict_sources(np.array([1.0, 2.0, np.nan, 3.0]), np.arange(4), 4, 4, 2, 0) == [2, 3]
    assert C.evict_sources(np.zeros(3), np.arange(3), 3, 3, 5, 1) == [0, 1, 2]


def test_acceptance_oracle_by_hand():
    #        0 -> 1 (a), 2 (b);  2 -> 3 (c), 4 (c);  1 -> 5 (d)
    par = np.array([-1, 0, 0, 2, 2, 1])
    draft = np.array([9, 10, 11, 12, 12, 13])
    assert C.accept(draft, np.array([11, 13, 12, 77, 78, 79]), par) == ([0, 2, 3], 77)
    assert C.accept(draft, np.array([10, 13, 12, 77, 78, 79]), par) == ([0, 1, 5], 79)
    assert C.accept(draft, np.array([99, 13, 12, 77, 78, 79]), par) == ([0], 99)
    assert C.accept(draft, np.array([11, 13, 12, 77, 78, 79]), np.array([-2, 0, 0, 2, 2, 1])) == ([], -1)


def test_fine_exponential_polynomial():
    # the constants of exp2_poly2_fine, evaluated as the kernel does, against 2^f on [-1/2, 1/2]
    src = open(os.path.join(os.path.dirname(B.__file__), "csrc", "rows_attention.cuh")).read()
    body = src[src.index("void exp2_poly2_fine("):]
    c = [np.float32(x) for x in re.findall(r"f2_pack\(([0-9.]+)f, ", body[:body.index("f2_unpack")])]
    assert len(c) == 6                                   # degree 5, highest first
    f = np.linspace(-0.5, 0.5, 100001).astype(np.float32)
    p = np.full_like(f, c[0])
    for k in c[1:]:
        p = (p.astype(np.float64) * f + k).astype(np.float32)      # one rounding per fused step
    assert np.abs(p / np.exp2(f.astype(np.float64)) - 1).max() < 2.4e-7
