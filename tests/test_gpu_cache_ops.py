"""GPU parity of the cache operators against their fp64 oracle.

Tolerances, per element.  A score is a sum of hd products accumulated in fp32,
off by at most ds = (hd + 8) 2^-23 max_j sum_d |q_d k_jd| / sqrt(hd) (twice
the half step per operation: an accumulator that truncates is covered too).
Each probability is then off by a factor 1 +- 2 ds (its own score and the sum's)
and the exponential's own error, and the sums over n keys add n 2^-23.  bf16
kernels store the probabilities in bf16 before the product with V (2^-8, half
a step) and may take the exponential from a cubic (2^-13); the accumulated
weights are fp32 throughout.  The result's own rounding is half a step of its
type."""
import numpy as np
import pytest
import torch

from helpers import GuardArena, f64
from llama_decoder_only_rmsnorm_b200 import binding as B
from oracle import cache_oracle as C

DEV = "cuda"
pytestmark = pytest.mark.gpu
G = None   # the running test's guard arena: outputs, caches and workspaces sit between guard bands
STATUS = 0  # status word the test expects to be set


@pytest.fixture(autouse=True)
def _gpu_state():
    global G, STATUS
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    B.llama3_set_kernel_path(0)
    G, STATUS = GuardArena(DEV), 0
    yield
    B.llama3_set_kernel_path(0)
    torch.cuda.synchronize()
    assert B.llama3_device_status() == STATUS, "device status word"
    G.check()


def dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def conf(H, KV, hd, dtype):
    return B.make_config(H * hd, H, KV, 4 * H * hd, dtype=dtype)


def randn(rng, shape, dtype, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dt(dtype))


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def workspace(n):
    # NaN patterns: nothing may be read before it is written
    return G.full((max(n, 16),), 0xFF, torch.uint8)


def out_bound(o, mag, dot, hd, keys, dtype):
    ds = (hd + 8) * 2.0 ** -23 * dot
    if dtype == "f32":
        return mag * (2.0 ** -20 + 4 * ds + keys * 2.0 ** -23) + np.abs(o) * 2.0 ** -24 + 1e-30
    return mag * (2.0 ** -8 + 2.0 ** -12 + 4 * ds + keys * 2.0 ** -23) * 1.01 + np.abs(o) * 2.0 ** -8 + 1e-30


def check(got, want, bound, what):
    assert got.shape == want.shape
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:4].tolist(), float(np.nanmax(err / bound)))


def make_tree(rng, T, shape, live=None):
    if shape == "chain":
        p = np.arange(T) - 1
    elif shape == "star":
        p = np.where(np.arange(T) == 0, -1, 0)
    elif shape == "roots":
        p = np.full(T, -1)
    else:
        p = np.array([-1] + [int(rng.integers(max(0, (t - 1) // 3), t)) for t in range(1, T)])
    if live is not None:
        p = np.where(np.arange(T) < live, p, -2)
    return p


HEADS = [(4, 2, 16, "f32"), (4, 2, 16, "bf16"), (8, 8, 32, "bf16"), (8, 4, 64, "f32"), (8, 4, 64, "bf16"),
         (8, 2, 96, "bf16"), (12, 4, 64, "bf16"), (16, 1, 128, "bf16"), (8, 2, 128, "bf16"), (6, 2, 96, "f32"),
         (5, 5, 128, "f32"), (20, 1, 64, "bf16")]


# ------------------------------------------------------------ tree attention
def run_tree(H, KV, hd, dtype, lens, T, parents, seed=1, extra=3, max_len=None, path=0, poison=True, stream=None):
    rng = np.random.default_rng(seed)
    Bn = len(lens)
    max_len = max(lens) if max_len is None else max_len
    cap = max(1, max_len + extra)
    q = randn(rng, (Bn, T, H, hd), dtype, 1.5)
    k, v = (randn(rng, (Bn, cap, KV, hd), dtype) for _ in range(2))
    kn, vn = (randn(rng, (Bn, T, KV, hd), dtype) for _ in range(2))
    if poison:
        for b in range(Bn):
            k[b, lens[b]:], v[b, lens[b]:] = float("nan"), float("inf")
            for t in range(T):
                if C.ancestors(parents[b], t) is None:
                    kn[b, t], vn[b, t], q[b, t] = float("nan"), float("-inf"), float("nan")
    cfg = conf(H, KV, hd, dtype)
    B.llama3_set_kernel_path(path)
    ws = workspace(B.llama3_tree_workspace_size(cfg, Bn, T, max_len))
    out = G.full((Bn, T, H * hd), 7.0, dt(dtype))
    B.llama3_attention_tree(cfg, q.to(DEV), k.to(DEV), v.to(DEV), cap, i32(lens), max_len, kn.to(DEV), vn.to(DEV),
                            i32(parents), Bn, T, out, ws, ws.numel(), stream)
    torch.cuda.synchronize()
    want, mag, dot = C.tree_attention(f64(q), f64(k), f64(v), lens, f64(kn), f64(vn), parents)
    keys = max(lens) + T
    check(f64(out).reshape(want.shape), want, out_bound(want, mag, dot, hd, keys, dtype), "tree")
    return out


@pytest.mark.parametrize("H,KV,hd,dtype", HEADS)
def test_tree_attention_head_layouts(H, KV, hd, dtype):
    rng = np.random.default_rng(7)
    lens = [130, 0, 257]
    par = np.stack([make_tree(rng, 13, "random", live) for live in (13, 9, 13)])
    run_tree(H, KV, hd, dtype, lens, 13, par)


@pytest.mark.parametrize("hd,dtype", [(64, "bf16"), (128, "bf16"), (96, "bf16"), (64, "f32")])
@pytest.mark.parametrize("T,shape,lens,max_len", [
    (1, "chain", [0], None), (1, "chain", [1, 1], None), (2, "star", [127, 128, 129], None),
    (33, "random", [640, 5], None), (64, "chain", [63], 300), (64, "random", [1025], None),
    (70, "roots", [64], None), (128, "random", [200, 0], 512), (256, "random", [31], None), (17, "star", [0, 0], 0)])
def test_tree_attention_sizes(hd, dtype, T, shape, lens, max_len):
    rng = np.random.default_rng(T)
    par = np.stack([make_tree(rng, T, shape) for _ in lens])
    run_tree(4, 2, hd, dtype, lens, T, par, seed=T + hd, max_len=max_len)


def test_tree_attention_long_cache_is_split():
    par = make_tree(np.random.default_rng(1), 5, "random")[None]
    run_tree(4, 1, 128, "bf16", [20011], 5, par)
    run_tree(2, 2, 64, "f32", [9001], 3, par[:, :3])


def test_tree_attention_plain_kernels_agree():
    par = make_tree(np.random.default_rng(2), 40, "random", 37)[None]
    run_tree(8, 2, 128, "bf16", [300], 40, par, path=1)


def test_tree_attention_all_padding_and_bad_parents():
    global STATUS
    par = np.full((2, 6), -3)
    run_tree(4, 2, 64, "bf16", [50, 0], 6, par)
    par = make_tree(np.random.default_rng(3), 6, "random")[None].copy()
    par[0, 4] = 5          # a parent behind its child: reported, and the node is padding
    run_tree(4, 2, 64, "bf16", [50], 6, par)
    STATUS = 1


def test_tree_attention_other_nodes_have_no_influence():
    # an infinity in a live node reaches the node and its descendants only
    H, KV, hd, T = 4, 2, 64, 6
    par = np.array([[-1, 0, 0, 1, 2, 2]])
    rng = np.random.default_rng(5)
    q, kn, vn = randn(rng, (1, T, H, hd), "bf16"), randn(rng, (1, T, KV, hd), "bf16"), randn(rng, (1, T, KV, hd), "bf16")
    k, v = (randn(rng, (1, 40, KV, hd), "bf16").to(DEV) for _ in range(2))
    cfg = conf(H, KV, hd, "bf16")
    outs = []
    for bad in (False, True):
        if bad:
            vn[0, 1], kn[0, 3] = float("inf"), float("nan")
        ws = workspace(B.llama3_tree_workspace_size(cfg, 1, T, 40))
        out = G.zeros((1, T, H * hd), torch.bfloat16)
        B.llama3_attention_tree(cfg, q.to(DEV), k, v, 40, i32([40]), 40, kn.to(DEV), vn.to(DEV), i32(par), 1, T, out,
                                ws, ws.numel())
        outs.append(f64(out)[0])
    np.testing.assert_array_equal(outs[0][[0, 2, 4, 5]], outs[1][[0, 2, 4, 5]])
    assert not np.isfinite(outs[1][[1, 3]]).all(-1).any()


def test_tree_attention_reports_a_length_outside():
    global STATUS
    cfg = conf(4, 2, 64, "bf16")
    rng = np.random.default_rng(6)
    q, kn, vn = (randn(rng, (2, 3, h, 64), "bf16").to(DEV) for h in (4, 2, 2))
    k, v = (randn(rng, (2, 20, 2, 64), "bf16").to(DEV) for _ in range(2))
    par = i32([[-1, 0, 1]] * 2)
    outs = []
    for lens in ([-4, 21], [0, 20]):   # clamped
        ws = workspace(B.llama3_tree_workspace_size(cfg, 2, 3, 20))
        out = G.zeros((2, 3, 256), torch.bfloat16)
        B.llama3_attention_tree(cfg, q, k, v, 20, i32(lens), 20, kn, vn, par, 2, 3, out, ws, ws.numel())
        outs.append(out)
    assert torch.equal(*outs)
    STATUS = 1


# -------------------------------------------------------- observed attention
def run_observe(H, KV, hd, dtype, lens, S, rows, seed=1, extra=2, max_len=None, path=0, in_place=False, win=True,
                null_lens=False, null_rows=False, positions=True):
    rng = np.random.default_rng(seed)
    Bn = len(lens)
    max_len = max(lens) if max_len is None else max_len
    cap = max_len + S + extra
    q = randn(rng, (Bn, S, H, hd), dtype, 1.5)
    k, v = (randn(rng, (Bn, cap, KV, hd), dtype) for _ in range(2))
    w_in = torch.from_numpy(rng.uniform(0, 4, (Bn, KV, cap)).astype(np.float32))
    for b in range(Bn):
        k[b, lens[b] + rows[b]:], v[b, lens[b] + rows[b]:] = float("nan"), float("-inf")
        q[b, rows[b]:] = float("nan")
        w_in[b, :, lens[b]:] = float("nan")
    cfg = conf(H, KV, hd, dtype)
    B.llama3_set_kernel_path(path)
    ws = workspace(B.llama3_observe_workspace_size(cfg, Bn, S, max_len))
    out = G.full((Bn, S, H * hd), 7.0, dt(dtype))
    before = w_in if in_place else torch.full((Bn, KV, cap), -7.0)
    w = G.to(before)
    slot_pos = G.full((Bn, KV, cap), -9, torch.int32)
    pos = [3 * n + 5 for n in lens]
    B.llama3_attention_observed(cfg, q.to(DEV), k.to(DEV), v.to(DEV), cap, Bn, S, None if null_lens else i32(lens),
                                None if null_rows else i32(rows), max_len, out,
                                (w if in_place else w_in.to(DEV)) if win else None, w,
                                i32(pos) if positions else None, slot_pos, ws, ws.numel())
    torch.cuda.synchronize()
    want, mag, dot, wts = C.observed_attention(f64(q), f64(k), f64(v), lens, rows, f64(w_in) if win else None)
    keys = max_len + S
    check(f64(out).reshape(want.shape), want, out_bound(want, mag, dot, hd, keys, dtype), "out")
    new = ~np.isnan(wts)
    base = np.where(new, f64(w_in) if win else 0.0, 0.0)
    base = np.where(np.isnan(base), 0.0, base)
    rel = 2.0 ** -20 + 4 * (hd + 8) * 2.0 ** -23 * dot.max() + (keys + S * H // KV) * 2.0 ** -23
    got = f64(w)
    wbound = np.where(new, (wts - base) * rel + np.abs(wts) * 2.0 ** -23 + 1e-30, 0.0)
    check(np.where(new, got, 0.0), np.where(new, wts, 0.0), wbound, "weights")
    np.testing.assert_array_equal(np.where(new, 0.0, got), np.where(new, 0.0, f64(before)))
    sp = slot_pos.cpu().numpy()
    for b in range(Bn):
        exp = np.full(cap, -9)
        exp[lens[b]:lens[b] + rows[b]] = (pos[b] if positions else lens[b]) + np.arange(rows[b])
        np.testing.assert_array_equal(sp[b], np.broadcast_to(exp, (KV, cap)))
    return out, w


@pytest.mark.parametrize("H,KV,hd,dtype", HEADS)
@pytest.mark.parametrize("S,rows", [(1, [1, 1, 0]), (37, [37, 0, 20])])
def test_observed_attention_head_layouts(H, KV, hd, dtype, S, rows):
    run_observe(H, KV, hd, dtype, [130, 3, 257], S, rows)


@pytest.mark.parametrize("H,KV,hd,dtype", [(4, 2, 64, "bf16"), (8, 2, 128, "bf16"), (3, 3, 96, "bf16"), (4, 2, 16, "f32")])
@pytest.mark.parametrize("S,lens,rows,max_len", [
    (1, [0], [1], None), (1, [0, 127], [1, 1], None), (1, [128, 5], [0, 1], 200), (2, [0], [2], None),
    (1, [2500], [1], None), (5, [1021], [5], None), (128, [0], [128], None), (129, [127], [129], None),
    (300, [0, 40], [300, 1], 60), (64, [64, 200], [33, 64], None), (520, [11], [520], None)])
def test_observed_attention_sizes(H, KV, hd, dtype, S, lens, rows, max_len):
    run_observe(H, KV, hd, dtype, lens, S, rows, seed=S + hd, max_len=max_len)


@pytest.mark.parametrize("S", [1, 20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_observed_attention_argument_forms(S, dtype):
    run_observe(4, 2, 64, dtype, [70, 70], S, [S, S], null_lens=True, null_rows=True, win=False, positions=False)
    run_observe(4, 2, 64, dtype, [70, 9], S, [S, 1], in_place=True)
    run_observe(4, 2, 64, dtype, [70, 9], S, [0, 0])


def test_observed_attention_plain_kernels_agree():
    run_observe(8, 2, 128, "bf16", [300, 7], 40, [33, 40], path=1)
    run_observe(8, 2, 128, "bf16", [300, 7], 1, [1, 1], path=1)


@pytest.mark.parametrize("S", [1, 200])
def test_observed_attention_is_deterministic(S):
    a = run_observe(8, 2, 128, "bf16", [400, 33], S, [S, S])
    b = run_observe(8, 2, 128, "bf16", [400, 33], S, [S, S])
    assert torch.equal(a[0], b[0])
    # entries that were written hold no NaN; the others hold the same fill
    assert torch.equal(a[1], b[1])


def test_observed_attention_reports_lengths_outside():
    global STATUS
    cfg = conf(4, 2, 64, "bf16")
    rng = np.random.default_rng(8)
    for S in (1, 6):
        q = randn(rng, (2, S, 4, 64), "bf16").to(DEV)
        k, v = (randn(rng, (2, 30, 2, 64), "bf16").to(DEV) for _ in range(2))
        outs = []
        for lens, rows in (([-1, 99], [S + 1, -1]), ([0, 24], [S, 0])):   # clamped
            ws = workspace(B.llama3_observe_workspace_size(cfg, 2, S, 24))
            out, w = G.zeros((2, S, 256), torch.bfloat16), G.zeros((2, 2, 30))
            B.llama3_attention_observed(cfg, q, k, v, 30, 2, S, i32(lens), i32(rows), 24, out, None, w, None, None, ws,
                                        ws.numel())
            outs.append((out, w))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    STATUS = 1


# ------------------------------------------------------------------ eviction
def run_evict(layers, KV, hd, dtype, lens, cap, budget, recent, in_place, seed=1, kind="spread", max_len=None):
    rng = np.random.default_rng(seed)
    Bn = len(lens)
    m = cap if max_len is None else max_len
    dst_cap = cap if in_place else min(budget, m) + 1
    src = []
    for _ in range(layers):
        w = np.exp(2.0 * rng.standard_normal((Bn, KV, cap))).astype(np.float32)
        if kind == "ties":
            w = rng.integers(0, 3, w.shape).astype(np.float32) - 1.0
            w[rng.random(w.shape) < 0.2] = -0.0
        elif kind == "special":
            w[rng.random(w.shape) < 0.1] = np.nan
            w[rng.random(w.shape) < 0.1] = np.inf
            w[rng.random(w.shape) < 0.1] = -np.inf
            w[rng.random(w.shape) < 0.1] = 1e-42
        pos = np.stack([[rng.permutation(cap) for _ in range(KV)] for _ in range(Bn)]).astype(np.int32)
        src.append(dict(k=randn(rng, (Bn, cap, KV, hd), dtype), v=randn(rng, (Bn, cap, KV, hd), dtype),
                        weights=torch.from_numpy(w), slot_pos=torch.from_numpy(pos)))
    positions = [max(n, 1) + 2 for n in lens]
    d_src = [{n: G.to(t) for n, t in c.items()} for c in src]
    d_dst = d_src if in_place else [
        dict(k=G.full((Bn, dst_cap, KV, hd), 3.0, dt(dtype)), v=G.full((Bn, dst_cap, KV, hd), 3.0, dt(dtype)),
             weights=G.full((Bn, KV, dst_cap), 3.0), slot_pos=G.full((Bn, KV, dst_cap), 3, torch.int32)) for _ in src]
    before = [{n: t.cpu().clone() for n, t in c.items()} for c in d_dst]
    cfg = conf(KV, KV, hd, dtype)
    ws = workspace(B.llama3_evict_workspace_size(cfg, layers, Bn, m, budget))
    d_lens = G.to(torch.tensor(lens, dtype=torch.int32))
    B.llama3_cache_evict(cfg, B.make_bounded_caches(d_src), cap, None if in_place else B.make_bounded_caches(d_dst),
                         dst_cap, Bn, d_lens, m, budget, recent, i32(positions), d_lens, ws, ws.numel())
    torch.cuda.synchronize()
    assert d_lens.tolist() == [min(n, budget) for n in lens]
    for s, d, old in zip(src, d_dst, before):
        want = {n: t.clone() for n, t in old.items()}
        for b in range(Bn):
            for g in range(KV):
                take = C.evict_sources(s["weights"][b, g].numpy(), s["slot_pos"][b, g].numpy(), lens[b], positions[b],
                                       budget, recent)
                n = len(take)
                for name in ("k", "v"):
                    want[name][b, :n, g] = s[name][b, take, g]
                for name in ("weights", "slot_pos"):
                    want[name][b, g, :n] = s[name][b, g, take]
        for name in want:
            # bit for bit, NaN included
            a, e = d[name].cpu().contiguous(), want[name].contiguous()
            assert torch.equal(a.view(torch.uint8), e.view(torch.uint8)), name


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
@pytest.mark.parametrize("layers,KV,hd,dtype,lens,cap,budget,recent", [
    (1, 1, 16, "f32", [9], 9, 4, 2), (2, 2, 64, "bf16", [40, 17, 0], 41, 16, 5), (1, 8, 128, "bf16", [1500], 1600, 300, 64),
    (1, 2, 96, "bf16", [1024, 1025], 1025, 1024, 0), (1, 2, 32, "bf16", [70, 3], 70, 1, 1),
    (1, 1, 16, "bf16", [200], 200, 100, 100), (1, 1, 64, "bf16", [3000, 2049], 3001, 2048, 100), (1, 1, 64, "f32", [5, 5], 8, 8, 8)])
def test_eviction(in_place, kind, layers, KV, hd, dtype, lens, cap, budget, recent):
    run_evict(layers, KV, hd, dtype, lens, cap, budget, recent, in_place, kind=kind)


def test_eviction_many_layers_and_long_rows():
    run_evict(35, 1, 16, "f32", [30, 12], 30, 10, 3, False)
    run_evict(35, 1, 16, "f32", [30, 12], 30, 10, 3, True)
    run_evict(1, 1, 16, "f32", [70001], 70001, 30000, 500, False, kind="ties")
    run_evict(1, 1, 16, "f32", [70001], 70001, 300, 50, True)


def test_eviction_into_a_smaller_cache_than_the_budget():
    run_evict(1, 2, 64, "bf16", [20, 7], 20, 64, 9, False, max_len=20)


# ---------------------------------------------------------------- acceptance
@pytest.mark.parametrize("layers,KV,hd,dtype,Bn,T,shape", [
    (1, 2, 16, "f32", 1, 1, "chain"), (3, 2, 64, "bf16", 5, 12, "random"), (70, 1, 16, "f32", 2, 5, "random"),
    (2, 8, 128, "bf16", 3, 64, "chain"), (1, 2, 96, "bf16", 2, 256, "random"), (1, 2, 64, "bf16", 4, 9, "star"),
    (1, 2, 64, "bf16", 2, 9, "roots")])
@pytest.mark.parametrize("extras", [False, True])
def test_acceptance_and_commit(layers, KV, hd, dtype, Bn, T, shape, extras):
    rng = np.random.default_rng(T * 31 + Bn)
    cap = 40 + T
    par = np.stack([make_tree(rng, T, shape, max(1, T - 3 * b)) for b in range(Bn)])
    if Bn > 2:
        par[1, 0] = -2          # a sequence without a tree
    draft, target = (rng.integers(0, 3, (Bn, T)) for _ in range(2))   # few tokens: many twins
    for b in range(Bn):         # and paths of some length: most nodes are followed by one of their children
        for t in range(T):
            if par[b, t] >= 0 and rng.random() < 0.9:
                target[b, par[b, t]] = draft[b, t]
    lens = rng.integers(0, 41, Bn)
    pos = lens + 100
    nodes = [dict(k=randn(rng, (Bn, T, KV, hd), dtype).to(DEV), v=randn(rng, (Bn, T, KV, hd), dtype).to(DEV))
             for _ in range(layers)]
    caches = [dict(k=G.full((Bn, cap, KV, hd), 2.0, dt(dtype)), v=G.full((Bn, cap, KV, hd), 2.0, dt(dtype)))
              for _ in range(layers)]
    if extras:
        for c in caches:
            c["weights"], c["slot_pos"] = G.full((Bn, KV, cap), 5.0), G.full((Bn, KV, cap), 5, torch.int32)
    path, acc, nxt = G.full((Bn, T), 9, torch.int32), G.full((Bn,), 9, torch.int32), G.full((Bn,), 9, torch.int32)
    d_lens, d_pos = G.to(torch.tensor(lens, dtype=torch.int32)), G.to(torch.tensor(pos, dtype=torch.int32))
    B.llama3_tree_accept(i32(draft), i32(target), i32(par), Bn, T, d_lens, path, acc, nxt, d_lens,
                         *((d_pos, d_pos) if extras else ()))
    cfg = conf(KV, KV, hd, dtype)
    B.llama3_tree_commit(cfg, B.make_bounded_caches(nodes), B.make_bounded_caches(caches), cap, Bn, T, path, acc,
                         d_lens, d_pos if extras else None)
    torch.cuda.synchronize()
    longest = 0
    for b in range(Bn):
        p, token = C.accept(draft[b], target[b], par[b])
        n = len(p)
        longest = max(longest, n)
        assert path[b].tolist() == p + [-1] * (T - n)
        assert (acc[b].item(), nxt[b].item(), d_lens[b].item()) == (n, token, lens[b] + n)
        assert d_pos[b].item() == pos[b] + (n if extras else 0)
        for nd, c in zip(nodes, caches):
            for name in ("k", "v"):
                assert torch.equal(c[name][b, lens[b]:lens[b] + n], nd[name][b, p])
                assert (c[name][b, :lens[b]] == 2).all() and (c[name][b, lens[b] + n:] == 2).all()
            if extras:
                w, sp = c["weights"][b].cpu().numpy(), c["slot_pos"][b].cpu().numpy()
                ew, ep = np.full(cap, 5.0), np.full(cap, 5)
                ew[lens[b]:lens[b] + n], ep[lens[b]:lens[b] + n] = 0.0, pos[b] + np.arange(n)
                np.testing.assert_array_equal(w, np.broadcast_to(ew, w.shape))
                np.testing.assert_array_equal(sp, np.broadcast_to(ep, sp.shape))
    assert longest > 1 or T < 8 or shape == "roots"   # small random trees may well confirm nothing


def test_commit_leaves_a_full_cache_alone():
    global STATUS
    cfg = conf(2, 2, 64, "bf16")
    nodes = [dict(k=torch.ones((1, 3, 2, 64), dtype=torch.bfloat16, device=DEV),
                  v=torch.ones((1, 3, 2, 64), dtype=torch.bfloat16, device=DEV))]
    caches = [dict(k=G.zeros((1, 4, 2, 64), torch.bfloat16), v=G.zeros((1, 4, 2, 64), torch.bfloat16))]
    for path, acc, lens in (([[0, 1, 2]], [3], [6]), ([[0, 1, 2]], [3], [2]), ([[0, 1, 2]], [4], [4]),
                            ([[0, 1, 2]], [-1], [2])):
        B.llama3_tree_commit(cfg, B.make_bounded_caches(nodes), B.make_bounded_caches(caches), 4, 1, 3, i32(path),
                             i32(acc), i32(lens))
        assert not caches[0]["k"].any() and not caches[0]["v"].any()
        assert B.llama3_device_status() == 1
    B.llama3_tree_commit(cfg, B.make_bounded_caches(nodes), B.make_bounded_caches(caches), 4, 1, 3, i32([[0, 3, -1]]),
                         i32([3]), i32([3]))   # nodes that do not exist are skipped
    assert caches[0]["k"][0, 0].all() and not caches[0]["k"][0, 1:].any()
    STATUS = 1
