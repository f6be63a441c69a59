"""Keys, queries and scores that are not finite, where the cache operators do look:
the softmax of a row over a NaN is NaN, and so is every weight that the row hands
out.  A NaN in the cache may not end as a number, whatever column of a tile the
key lies in and however the row's keys are cut into pieces.  What does not see the
value keeps its bits."""
import numpy as np
import pytest
import torch

import test_gpu_cache_ops as ops
from llama_decoder_only_rmsnorm_b200 import binding as B
from test_gpu_cache_ops import _gpu_state  # noqa: F401  (the guard arena and the status check)

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")
FORMS = [("bf16", 0, 64), ("bf16", 0, 128), ("bf16", 1, 64), ("f32", 0, 32)]


class Call:
    """Inputs of one call; tree(), observe() run it on what they hold now."""

    def __init__(self, Bn, T, H, KV, hd, dtype, path, n, seed=1, cap=None):
        rng = np.random.default_rng(seed)
        self.shape, self.dtype, self.n = (Bn, T, H, KV, hd), dtype, n
        self.cap = n + T if cap is None else cap
        one = lambda *s: ops.randn(rng, (1,) + s, dtype).to(DEV).repeat((Bn,) + (1,) * len(s))   # sequences alike
        self.q, self.kn, self.vn = one(T, H, hd), one(T, KV, hd), one(T, KV, hd)
        self.k, self.v = one(self.cap, KV, hd), one(self.cap, KV, hd)
        self.par = ops.i32(np.tile(np.arange(T) - 1, (Bn, 1)))
        self.cfg = ops.conf(H, KV, hd, dtype)
        B.llama3_set_kernel_path(path)

    def tree(self):
        Bn, T, H, KV, hd = self.shape
        ws = ops.workspace(B.llama3_tree_workspace_size(self.cfg, Bn, T, self.n))
        out = ops.G.full((Bn, T, H * hd), 7.0, ops.dt(self.dtype))
        B.llama3_attention_tree(self.cfg, self.q, self.k, self.v, self.cap, ops.i32([self.n] * Bn), self.n, self.kn,
                                self.vn, self.par, Bn, T, out, ws, ws.numel())
        return out.view(Bn, T, KV, H // KV * hd).float().cpu()

    def observe(self):
        Bn, T, H, KV, hd = self.shape
        ws = ops.workspace(B.llama3_observe_workspace_size(self.cfg, Bn, T, self.n))
        out = ops.G.full((Bn, T, H * hd), 7.0, ops.dt(self.dtype))
        w = ops.G.full((Bn, KV, self.cap), 7.0)
        B.llama3_attention_observed(self.cfg, self.q, self.k, self.v, self.cap, Bn, T, ops.i32([self.n] * Bn), None,
                                    self.n, out, None, w, None, None, ws, ws.numel())
        return out.view(Bn, T, KV, H // KV * hd).float().cpu(), w.cpu()


@pytest.mark.parametrize("dtype,path,hd", FORMS)
@pytest.mark.parametrize("T", [2, 40])
def test_a_key_that_is_not_a_number_reaches_every_row_of_the_tree(dtype, path, hd, T):
    n = 290                                  # two whole key tiles and a part; sequence b has its NaN in key b
    c = Call(n, T, 8, 2, hd, dtype, path, n)
    clean = c.tree()
    at = torch.arange(n, device=DEV)
    c.k[at, at, 0, at % hd] = NAN
    out = c.tree()
    assert torch.isnan(out[:, :, 0]).all()
    assert torch.equal(out[:, :, 1], clean[:, :, 1]) and torch.isfinite(clean).all()


@pytest.mark.parametrize("dtype,path,hd", FORMS)
@pytest.mark.parametrize("T", [1, 3, 40])
def test_a_key_that_is_not_a_number_reaches_rows_and_weights(dtype, path, hd, T):
    n = 290
    c = Call(n, T, 8, 2, hd, dtype, path, n)
    out0, w0 = c.observe()
    at = torch.arange(n, device=DEV)
    c.k[at, at, 0, at % hd] = NAN
    out, w = c.observe()
    assert torch.isnan(out[:, :, 0]).all() and torch.isnan(w[:, 0]).all()
    assert torch.equal(out[:, :, 1], out0[:, :, 1]) and torch.equal(w[:, 1], w0[:, 1])
    assert torch.isfinite(out0).all() and torch.isfinite(w0).all()


@pytest.mark.parametrize("dtype,path,hd", FORMS)
def test_a_key_of_the_chunk_that_is_not_a_number_reaches_the_rows_behind_it(dtype, path, hd):
    T, n = 40, 200
    c = Call(T, T, 8, 2, hd, dtype, path, n)
    out0, w0 = c.observe()
    at = torch.arange(T, device=DEV)
    c.k[at, n + at, 0, 0] = NAN               # sequence b: the chunk's key b, seen by the rows from b on
    out, w = c.observe()
    for b in range(T):
        assert torch.equal(out[b, :b], out0[b, :b]), b
        assert torch.isnan(out[b, b:, 0]).all() and torch.equal(out[b, b:, 1], out0[b, b:, 1]), b
    assert torch.isnan(w[:, 0]).all() and torch.equal(w[:, 1], w0[:, 1])


@pytest.mark.parametrize("dtype,path,hd", FORMS)
@pytest.mark.parametrize("T", [1, 70])
def test_a_query_that_is_not_a_number_reaches_the_weights_it_hands_out(dtype, path, hd, T):
    H, KV, n = 8, 2, 300
    c = Call(T * 4, T, H, KV, hd, dtype, path, n)
    out0, w0 = c.observe()
    for b in range(T * 4):                   # one head of one position per sequence
        c.q[b, b // 4, b % 4, 0] = NAN
    out, w = c.observe()
    heads = lambda o: o.view(T * 4, T, H, hd)
    for b in range(T * 4):
        t, h = b // 4, b % 4
        assert torch.isnan(heads(out)[b, t, h]).all(), b
        rest = torch.ones((T, H), dtype=torch.bool)
        rest[t, h] = False
        assert torch.equal(heads(out)[b][rest], heads(out0)[b][rest]), b
        assert torch.isnan(w[b, 0, :n + t + 1]).all() and torch.equal(w[b, 0, n + t + 1:], w0[b, 0, n + t + 1:]), b
    assert torch.equal(w[:, 1], w0[:, 1])


@pytest.mark.parametrize("dtype,path,hd", FORMS)
@pytest.mark.parametrize("where", [slice(0, 1300), slice(2000, 3400), slice(0, 5000)])
def test_pieces_of_nothing_but_such_keys_count(dtype, path, hd, where):
    # whole pieces of the row (a CTA's share of the keys) hold no number at all
    for KV, T in ((1, 1), (1, 5), (2, 3)):
        c = Call(1, T, 2 * KV, KV, hd, dtype, path, 5000)
        c.k[0, where, 0] = NAN
        tree = c.tree()
        out, w = c.observe()
        assert torch.isnan(tree[:, :, 0]).all() and torch.isnan(out[:, :, 0]).all() and torch.isnan(w[:, 0]).all()
        assert torch.isfinite(tree[:, :, 1:]).all() and torch.isfinite(out[:, :, 1:]).all()
        assert torch.isfinite(w[:, 1:]).all()


@pytest.mark.parametrize("dtype,path,hd", FORMS)
def test_infinite_scores(dtype, path, hd):
    # +inf: inf - inf, so NaN.  -inf: the key takes no part; 3e38 is finite in both types, its score is not
    n = 290
    c = Call(n, 3, 8, 2, hd, dtype, path, n)
    c.q.fill_(1.5)
    at = torch.arange(n, device=DEV)
    plain = c.k.clone()
    c.k[at, at, 0] = 3e38
    out, w = c.observe()
    assert torch.isnan(c.tree()[:, :, 0]).all() and torch.isnan(out[:, :, 0]).all() and torch.isnan(w[:, 0]).all()
    c.k.copy_(plain)
    c.k[at, at, 0] = -3e38
    tree, (out, w) = c.tree(), c.observe()
    assert torch.isfinite(tree).all() and torch.isfinite(out).all() and torch.isfinite(w).all()
    # of 2^-126 at most per row and head, the floor of the polynomial
    assert (w[at.cpu(), 0, at.cpu()] <= 12 * 2.0 ** -126).all()
    c.v[at, at, 0] = 1e4                      # the key's value has no influence
    assert torch.equal(c.tree(), tree) and torch.equal(c.observe()[0], out)
