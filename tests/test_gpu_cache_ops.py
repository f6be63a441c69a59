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


@pytest.mark.parametrize("H,KV,hd,dtype", [(100, 1, 32, "bf16"), (64, 1, 16, "f32"), (33, 1, 96, "bf16"),
                                           (128, 1, 128, "bf16")])
def test_many_heads_of_one_kv_head(H, KV, hd, dtype):
    par = make_tree(np.random.default_rng(9), 3, "random")[None]
    run_tree(H, KV, hd, dtype, [140], 3, par)
    run_observe(H, KV, hd, dtype, [140], 3, [2])
    run_observe(H, KV, hd, dtype, [140], 1, [1])


def test_tree_attention_long_cache_is_split():
    par = make_tree(np.random.default_rng(1), 5, "random")[None]
    run_tree(4, 1, 128, "bf16", [20011], 5, par)
    run_tree(2, 2, 64, "f32", [9001], 3, par[:, :3])


@pytest.mark.parametrize("H,KV,hd,dtype", [(16, 1, 128, "bf16"), (4, 2, 64, "bf16"), (2, 1, 16, "f32"), (3, 1, 96, "bf16")])
def test_one_long_cache_of_few_heads(H, KV, hd, dtype):
    # dozens of pieces per row; a second, short sequence has none or one
    par = np.stack([make_tree(np.random.default_rng(4), 6, "random", n) for n in (6, 3)])
    for lens in ([12000], [15001, 100], [9000, 0]):
        run_tree(H, KV, hd, dtype, lens, 6, par[:len(lens)])
        run_observe(H, KV, hd, dtype, lens, 1, [1] * len(lens))
        run_observe(H, KV, hd, dtype, lens, 5, [5, 2][:len(lens)])


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


def test_eviction_in_place_shortens_the_lengths_it_reads():
    # more blocks than run at once, and kv_lens_out is kv_lens: those that start late see the new lengths
    run_evict(32, 2, 128, "bf16", [2048, 1900], 2048, 700, 100, True)


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


# ------------------------------------------------------------ ways of calling
def _tree_call(seed, lens=(300, 17), T=12, H=8, KV=2, hd=128):
    """A tree attention call and its output: call(stream)."""
    rng = np.random.default_rng(seed)
    Bn, max_len = len(lens), max(lens)
    par = i32(np.stack([make_tree(rng, T, "random") for _ in lens]))
    q, kn, vn = (randn(rng, (Bn, T, h, hd), "bf16").to(DEV) for h in (H, KV, KV))
    k, v = (randn(rng, (Bn, max_len, KV, hd), "bf16").to(DEV) for _ in range(2))
    cfg, d_lens = conf(H, KV, hd, "bf16"), i32(lens)
    ws = workspace(B.llama3_tree_workspace_size(cfg, Bn, T, max_len))
    out = G.zeros((Bn, T, H * hd), torch.bfloat16)
    return lambda stream=None: B.llama3_attention_tree(cfg, q, k, v, max_len, d_lens, max_len, kn, vn, par, Bn, T, out,
                                                       ws, ws.numel(), stream), out


def _observe_call(seed, S, lens=(300, 17), H=8, KV=2, hd=128):
    rng = np.random.default_rng(seed)
    Bn, max_len = len(lens), max(lens)
    cap = max_len + S
    q = randn(rng, (Bn, S, H, hd), "bf16").to(DEV)
    k, v = (randn(rng, (Bn, cap, KV, hd), "bf16").to(DEV) for _ in range(2))
    cfg, d_lens = conf(H, KV, hd, "bf16"), i32(lens)
    ws = workspace(B.llama3_observe_workspace_size(cfg, Bn, S, max_len))
    out, w = G.zeros((Bn, S, H * hd), torch.bfloat16), G.zeros((Bn, KV, cap))
    return lambda stream=None: B.llama3_attention_observed(cfg, q, k, v, cap, Bn, S, d_lens, None, max_len, out, None, w,
                                                           None, None, ws, ws.numel(), stream), (out, w)


def test_two_streams_at_once_give_what_one_gives():
    calls = [_tree_call(1), _observe_call(2, 1), _tree_call(3, (1000,), 64), _observe_call(4, 150)]
    for call, _ in calls:
        call()
    torch.cuda.synchronize()
    flat = lambda o: [t.clone() for t in (o if isinstance(o, tuple) else (o,))]
    want = [flat(o) for _, o in calls]
    for _, o in calls:
        for t in (o if isinstance(o, tuple) else (o,)):
            t.zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(3):
        for (call, _), s in zip(calls, streams):
            call(s)
    torch.cuda.synchronize()
    for (_, o), w in zip(calls, want):
        for a, b in zip(flat(o), w):
            assert torch.equal(a, b)


def test_ordinary_launches_give_the_same():
    for make in (lambda: _tree_call(5), lambda: _observe_call(6, 1), lambda: _observe_call(7, 70)):
        call, o = make()
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in (o if isinstance(o, tuple) else (o,))]
        old = B.llama3_set_programmatic_launch(0)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            B.llama3_set_programmatic_launch(old)
        assert all(torch.equal(a, b) for a, b in zip(o if isinstance(o, tuple) else (o,), want))


def test_rows_far_behind_4_gib():
    # the last sequence's rows begin 8 GiB into each cache, and the capacity bounds every plan
    H, KV, hd, cap, Bn, n = 8, 8, 128, 1 << 20, 5, 90
    rng = np.random.default_rng(11)
    k, v = (torch.zeros((Bn, cap, KV, hd), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rows = [randn(rng, (n + 8, KV, hd), "bf16") for _ in range(2)]
    k[-1, :n + 8], v[-1, :n + 8] = rows[0].to(DEV), rows[1].to(DEV)
    lens = [0] * (Bn - 1) + [n]
    cfg, d_lens, T = conf(H, KV, hd, "bf16"), i32(lens), 4
    par = np.tile(make_tree(rng, T, "chain"), (Bn, 1))
    q = randn(rng, (Bn, T, H, hd), "bf16")
    kn, vn = (randn(rng, (Bn, T, KV, hd), "bf16") for _ in range(2))
    max_len = cap - T
    ws = workspace(B.llama3_tree_workspace_size(cfg, Bn, T, max_len))
    out = G.zeros((Bn, T, H * hd), torch.bfloat16)
    B.llama3_attention_tree(cfg, q.to(DEV), k, v, cap, d_lens, max_len, kn.to(DEV), vn.to(DEV), i32(par), Bn, T, out, ws,
                            ws.numel())
    want, mag, dot = C.tree_attention(f64(q[-1:]), f64(rows[0][None]), f64(rows[1][None]), [n], f64(kn[-1:]),
                                      f64(vn[-1:]), par[-1:])
    check(f64(out[-1]).reshape(want[0].shape), want[0], out_bound(want, mag, dot, hd, n + T, "bf16")[0], "tree")
    for S in (1, T):
        ws = workspace(B.llama3_observe_workspace_size(cfg, Bn, S, max_len))
        w = torch.zeros((Bn, KV, cap), device=DEV)
        out = G.zeros((Bn, S, H * hd), torch.bfloat16)
        live = [0] * (Bn - 1) + [S]
        B.llama3_attention_observed(cfg, q[:, :S].contiguous().to(DEV), k, v, cap, Bn, S, d_lens, i32(live), max_len,
                                    out, None, w, None, None, ws, ws.numel())
        want, mag, dot, wts = C.observed_attention(f64(q[-1:, :S]), f64(rows[0][None]), f64(rows[1][None]), [n], [S],
                                                   None)
        check(f64(out[-1]).reshape(want[0].shape), want[0], out_bound(want, mag, dot, hd, n + S, "bf16")[0], "out")
        np.testing.assert_allclose(f64(w[-1, :, :n + S]), wts[0, :, :n + S], rtol=2e-5, atol=1e-9)
        assert not w[-1, :, n + S:].any() and not w[:-1].any()
    # eviction of the last sequence into its own place, and a path committed behind it
    w = torch.zeros((Bn, KV, cap), device=DEV)
    pos = torch.zeros((Bn, KV, cap), dtype=torch.int32, device=DEV)
    wr = rng.uniform(0, 1, (KV, n)).astype(np.float32)
    w[-1, :, :n], pos[-1, :, :n] = torch.from_numpy(wr).to(DEV), torch.arange(n, dtype=torch.int32, device=DEV)
    cache = B.make_bounded_caches([dict(k=k, v=v, weights=w, slot_pos=pos)])
    budget, recent, d_pos = 40, 10, i32([n] * Bn)
    ws = workspace(B.llama3_evict_workspace_size(cfg, 1, Bn, cap, budget))
    B.llama3_cache_evict(cfg, cache, cap, None, 0, Bn, d_lens, cap, budget, recent, d_pos, d_lens, ws, ws.numel())
    assert d_lens.tolist() == [0] * (Bn - 1) + [budget]
    for g in range(KV):
        take = C.evict_sources(wr[g], np.arange(n), n, n, budget, recent)
        assert torch.equal(k[-1, :budget, g].cpu(), rows[0][take, g]) and torch.equal(v[-1, :budget, g].cpu(), rows[1][take, g])
        assert pos[-1, g, :budget].tolist() == take
    nodes = B.make_bounded_caches([dict(k=kn.to(DEV), v=vn.to(DEV))])
    keep = nodes, kn.to(DEV), vn.to(DEV)
    nodes = B.make_bounded_caches([dict(k=keep[1], v=keep[2])])
    d_lens += 2
    B.llama3_tree_commit(cfg, nodes, cache, cap, Bn, T, i32([[0, 2, -1, -1]] * Bn), i32([2] * Bn), d_lens)
    assert torch.equal(k[-1, budget:budget + 2].cpu(), kn[-1, [0, 2]]) and torch.equal(v[0, :2].cpu(), vn[0, [0, 2]])


# ----------------------------------------------------- all of them, as they are used
class Bounded:
    """Two layers of bounded caches driven as a drafting, evicting decoder drives
    them; what the model's projections would give is drawn at random."""
    H, KV, HD, L, BN, CAP, T = 8, 2, 64, 2, 3, 96, 9

    def __init__(self, dtype, seed):
        self.rng, self.dtype = np.random.default_rng(seed), dtype
        self.cfg = conf(self.H, self.KV, self.HD, dtype)
        shape = (self.BN, self.CAP, self.KV, self.HD)
        self.layers = [dict(k=G.full(shape, float("nan"), dt(dtype)), v=G.full(shape, float("nan"), dt(dtype)),
                            weights=G.full((self.BN, self.KV, self.CAP), float("nan")),
                            slot_pos=G.full((self.BN, self.KV, self.CAP), -1, torch.int32)) for _ in range(self.L)]
        self.caches = B.make_bounded_caches(self.layers)
        self.lens, self.pos = G.zeros((self.BN,), torch.int32), G.zeros((self.BN,), torch.int32)
        cfg = self.cfg
        n = max(B.llama3_observe_workspace_size(cfg, self.BN, 40, self.CAP - 40),
                B.llama3_observe_workspace_size(cfg, self.BN, 1, self.CAP - 1),
                B.llama3_tree_workspace_size(cfg, self.BN, self.T, self.CAP),
                B.llama3_evict_workspace_size(cfg, self.L, self.BN, self.CAP, 24))
        self.ws = workspace(n)

    def draw(self, S):
        return [[randn(self.rng, (self.BN, S, h, self.HD), self.dtype).to(DEV) for h in (self.H, self.KV, self.KV)]
                for _ in range(self.L)]

    def observe(self, qkv, rows, out):
        S = qkv[0][0].shape[1]
        lens = self.lens.tolist()
        for (q, k, v), c, o in zip(qkv, self.layers, out):
            for b in range(self.BN):
                c["k"][b, lens[b]:lens[b] + rows[b]] = k[b, :rows[b]]
                c["v"][b, lens[b]:lens[b] + rows[b]] = v[b, :rows[b]]
            B.llama3_attention_observed(self.cfg, q, c["k"], c["v"], self.CAP, self.BN, S, self.lens, i32(rows),
                                        self.CAP - S, o, c["weights"], c["weights"], self.pos, c["slot_pos"], self.ws,
                                        self.ws.numel())
        self.lens += i32(rows)
        self.pos += i32(rows)

    def evict(self, budget, recent):
        B.llama3_cache_evict(self.cfg, self.caches, self.CAP, None, 0, self.BN, self.lens, self.CAP, budget, recent,
                             self.pos, self.lens, self.ws, self.ws.numel())

    def tree(self, qkv, par, out):
        for (q, k, v), c, o in zip(qkv, self.layers, out):
            B.llama3_attention_tree(self.cfg, q, c["k"], c["v"], self.CAP, self.lens, self.CAP, k, v, par, self.BN,
                                    self.T, o, self.ws, self.ws.numel())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_drafting_decoder_with_bounded_caches(dtype):
    m = Bounded(dtype, 21)
    KV, BN, T = m.KV, m.BN, m.T
    out_t = lambda S: [G.zeros((BN, S, m.H * m.HD), dt(dtype)) for _ in range(m.L)]
    mirror = [[dict(k=[], v=[], pos=[[] for _ in range(KV)]) for _ in range(BN)] for _ in range(m.L)]   # rows per head
    seen = [0] * BN

    def rows_of(l, b):   # the mirror as [1, n, KV, hd]
        c = mirror[l][b]
        pack = lambda x: np.stack([np.stack(r) for r in x])[None] if x else np.zeros((1, 0, KV, m.HD))
        return pack(c["k"]), pack(c["v"])

    def step_observe(S, rows):
        qkv, out = m.draw(S), out_t(S)
        before = [f64(c["weights"]) for c in m.layers]
        lens = [len(mirror[0][b]["k"]) for b in range(BN)]
        m.observe(qkv, rows, out)
        for l, (q, k, v) in enumerate(qkv):
            for b in range(BN):
                for t in range(rows[b]):
                    mirror[l][b]["k"].append(f64(k[b, t]))
                    mirror[l][b]["v"].append(f64(v[b, t]))
                    for g in range(KV):
                        mirror[l][b]["pos"][g].append(seen[b] + t)
                kk, vv = rows_of(l, b)
                want, mag, dot, w = C.observed_attention(f64(q[b:b + 1]), kk, vv, [lens[b]], [rows[b]],
                                                         before[l][b:b + 1, :, :kk.shape[1]])
                check(f64(out[l][b]).reshape(want[0].shape), want[0],
                      out_bound(want, mag, dot, m.HD, kk.shape[1], dtype)[0], "out")
                np.testing.assert_allclose(f64(m.layers[l]["weights"][b, :, :kk.shape[1]]), w[0], rtol=2e-5, atol=1e-7)
        for b in range(BN):
            seen[b] += rows[b]

    def step_evict(budget, recent):
        lens = [len(mirror[0][b]["k"]) for b in range(BN)]
        weights = [c["weights"].cpu().numpy() for c in m.layers]   # the device's own sums decide
        m.evict(budget, recent)
        for l in range(m.L):
            for b in range(BN):
                c, n = mirror[l][b], min(lens[b], budget)
                new_k, new_v = [np.zeros((KV, m.HD)) for _ in range(n)], [np.zeros((KV, m.HD)) for _ in range(n)]
                for g in range(KV):
                    take = C.evict_sources(weights[l][b, g], c["pos"][g], lens[b], seen[b], budget, recent)
                    for i, j in enumerate(take):
                        new_k[i][g], new_v[i][g] = c["k"][j][g], c["v"][j][g]
                    c["pos"][g] = [c["pos"][g][j] for j in take]
                c["k"], c["v"] = new_k, new_v

    def step_tree(live):
        qkv, out = m.draw(T), out_t(T)
        par = np.stack([make_tree(m.rng, T, "random", n) for n in live])
        m.tree(qkv, i32(par), out)
        draft, target = m.rng.integers(0, 3, (BN, T)), m.rng.integers(0, 3, (BN, T))
        path, acc, nxt = (G.zeros(s, torch.int32) for s in ((BN, T), (BN,), (BN,)))
        B.llama3_tree_accept(i32(draft), i32(target), i32(par), BN, T, m.lens, path, acc, nxt, m.lens, m.pos, m.pos)
        nodes = B.make_bounded_caches([dict(k=k, v=v) for _, k, v in qkv])
        B.llama3_tree_commit(m.cfg, nodes, m.caches, m.CAP, BN, T, path, acc, m.lens, m.pos)
        for b in range(BN):
            p, token = C.accept(draft[b], target[b], par[b])
            assert path[b, :len(p)].tolist() == p and nxt[b].item() == token
            for l, (q, k, v) in enumerate(qkv):
                kk, vv = rows_of(l, b)
                want, mag, dot = C.tree_attention(f64(q[b:b + 1]), kk, vv, [kk.shape[1]], f64(k[b:b + 1]), f64(v[b:b + 1]),
                                                  par[b:b + 1])
                check(f64(out[l][b]).reshape(want[0].shape), want[0],
                      out_bound(want, mag, dot, m.HD, kk.shape[1] + T, dtype)[0], "tree")
                for i, t in enumerate(p):
                    mirror[l][b]["k"].append(f64(k[b, t]))
                    mirror[l][b]["v"].append(f64(v[b, t]))
                    for g in range(KV):
                        mirror[l][b]["pos"][g].append(seen[b] + i)
            seen[b] += len(p)

    step_observe(40, [40, 23, 31])      # padded prompts
    step_evict(24, 6)
    for live in ([9, 4, 0], [9, 9, 7]):
        step_tree(live)
        step_observe(1, [1, 1, 0])
    step_evict(24, 6)
    step_observe(1, [1, 1, 1])
    for l, c in enumerate(m.layers):
        for b in range(BN):
            n = len(mirror[l][b]["k"])
            assert m.lens[b].item() == n and m.pos[b].item() == seen[b]
            np.testing.assert_array_equal(f64(c["k"][b, :n]), rows_of(l, b)[0][0])
            np.testing.assert_array_equal(f64(c["v"][b, :n]), rows_of(l, b)[1][0])
            for g in range(KV):
                assert c["slot_pos"][b, g, :n].tolist() == mirror[l][b]["pos"][g]
            assert torch.isfinite(c["weights"][b, :, :n]).all()


def test_a_verification_step_replays_from_a_graph():
    # one captured step (tree attention, acceptance, commit, eviction), replayed as the caches grow and shrink
    def steps(m, graph):
        qkv = m.draw(m.T)
        par = i32(np.stack([make_tree(m.rng, m.T, "random", n) for n in (9, 7, 9)]))
        draft, target = (i32(m.rng.integers(0, 2, (m.BN, m.T))) for _ in range(2))
        path, acc, nxt = (G.zeros(s, torch.int32) for s in ((m.BN, m.T), (m.BN,), (m.BN,)))
        out = [G.zeros((m.BN, m.T, m.H * m.HD), torch.bfloat16) for _ in range(m.L)]
        nodes = B.make_bounded_caches([dict(k=k, v=v) for _, k, v in qkv])

        def one():
            m.tree(qkv, par, out)
            B.llama3_tree_accept(draft, target, par, m.BN, m.T, m.lens, path, acc, nxt, m.lens, m.pos, m.pos)
            B.llama3_tree_commit(m.cfg, nodes, m.caches, m.CAP, m.BN, m.T, path, acc, m.lens, m.pos)
            m.evict(24, 6)

        results = []
        if graph:
            state = [t.clone() for c in m.layers for t in c.values()] + [m.lens.clone(), m.pos.clone()]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                one()
            torch.cuda.current_stream().wait_stream(side)
            for t, old in zip([t for c in m.layers for t in c.values()] + [m.lens, m.pos], state):
                t.copy_(old)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                one()
        for _ in range(5):
            g.replay() if graph else one()
            torch.cuda.synchronize()
            results.append([t.clone() for t in out + [path, acc, nxt, m.lens, m.pos]])
        results.append([c[n][b, :x] if n in "kv" else c[n][b, :, :x] for c in m.layers for n in c
                        for b, x in enumerate(m.lens.tolist())])
        return results

    runs = []
    for graph in (False, True):
        m = Bounded("bf16", 33)
        m.observe(m.draw(40), [40, 23, 31], [G.zeros((m.BN, 40, m.H * m.HD), torch.bfloat16) for _ in range(m.L)])
        m.evict(24, 6)
        runs.append(steps(m, graph))
    for a, b in zip(*runs):
        assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
