"""The cache operators' variants that are chosen by size: each size here crosses the
border of one rule, which is asserted from the number of SMs, against the fp64
oracle with the tolerances of test_gpu_cache_ops."""
import numpy as np
import pytest
import torch

import test_gpu_cache_ops as ops
from test_gpu_cache_ops import _gpu_state  # noqa: F401  (the guard arena and the status check)

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def trees(seed, lives, T):
    rng = np.random.default_rng(seed)
    return np.stack([ops.make_tree(rng, T, "random", n) for n in lives])


# ---- tree attention: the joining kernel takes two or four heads of a node per warp
@pytest.mark.parametrize("H,KV,hd,dtype", [(16, 4, 64, "bf16"), (8, 1, 128, "bf16"), (8, 2, 32, "f32")])
def test_tree_joins_of_four_heads_per_warp(H, KV, hd, dtype):
    T, rep = 48, H // KV
    Bn = -(-64 * sms() // (T * H)) + 1
    assert rep % 4 == 0 and Bn * T * H >= 64 * sms()
    lens = [(37 * b) % 301 for b in range(Bn)]       # 0 among them
    ops.run_tree(H, KV, hd, dtype, lens, T, trees(1, [T - b % 5 for b in range(Bn)], T))


@pytest.mark.parametrize("H,KV,hd,dtype", [(8, 4, 64, "bf16"), (12, 2, 96, "bf16"), (8, 4, 16, "f32")])
def test_tree_joins_of_two_heads_per_warp(H, KV, hd, dtype):
    T, rep = 48, H // KV
    Bn = -(-32 * sms() // (T * H)) + 1
    rows = Bn * T * H
    assert rep % 2 == 0 and rows >= 32 * sms() and (rep % 4 != 0 or rows < 64 * sms())
    lens = [(41 * b + 5) % 290 for b in range(Bn)]
    ops.run_tree(H, KV, hd, dtype, lens, T, trees(2, [T - b % 7 for b in range(Bn)], T))


# ---- tree attention: two row tiles per CTA, out of much work; the length bound decides
@pytest.mark.parametrize("H,KV,hd", [(4, 2, 64), (8, 2, 96), (4, 4, 128), (6, 2, 32)])
@pytest.mark.parametrize("T,lens", [(160, [640, 0, 131]), (256, [1000, 129, 5]), (200, [127, 128, 2500])])
def test_tree_of_two_row_tiles_per_cta(H, KV, hd, T, lens):
    rep = H // KV
    tiles = -(-T // (128 // rep))                    # odd for some: the last group has one tile
    max_len = 128 * (16 * sms() // (len(lens) * KV * tiles) + 1)
    assert tiles > 1 and len(lens) * KV * tiles * (max_len // 128) > 16 * sms()
    ops.run_tree(H, KV, hd, "bf16", lens, T, trees(3, [T, T - 30, T // 2], T), max_len=max(max_len, max(lens)))


def test_tree_of_two_row_tiles_per_cta_over_a_long_cache():
    # one sequence: every group of tiles is cut into many pieces
    T, max_len = 130, 128 * (16 * sms() // 4 + 1)    # 2 KV heads of 2 tiles
    ops.run_tree(2, 2, 64, "bf16", [14001], T, trees(4, [T], T), max_len=max_len)


def test_nothing_cached_under_a_large_bound():
    for H, KV, hd, dtype in ((8, 2, 64, "bf16"), (4, 1, 128, "bf16"), (4, 2, 16, "f32")):
        ops.run_tree(H, KV, hd, dtype, [0, 0], 9, trees(5, [9, 4], 9), max_len=40000)
        ops.run_observe(H, KV, hd, dtype, [0, 0], 3, [3, 0], max_len=20000)


# ---- pieces that a launch of their own joins, with two row tiles per CTA
@pytest.mark.parametrize("S,rows", [(9, 9), (17, 16), (16, 3)])
def test_long_chunks_of_one_kv_head_fold_pairs_of_tiles(S, rows):
    H, n = 16, 128 * 80
    assert min(sms(), n // 128 + 1) > 64 and S * H > 128
    ops.run_observe(H, 1, 64, "bf16", [n + 5], S, [rows])


# ---- chunks of several groups and of many key tiles
@pytest.mark.parametrize("H,KV,hd,dtype", [(4, 2, 64, "bf16"), (4, 1, 128, "bf16"), (2, 2, 96, "f32")])
def test_long_chunks(H, KV, hd, dtype):
    ops.run_observe(H, KV, hd, dtype, [77, 0], 1337, [1337, 640], max_len=901)


# ---- eviction: many rows take blocks of 256 threads
def many(layers, Bn, KV, cap):
    assert min(layers, 32) * Bn * KV >= 2 * sms() and cap <= 8192


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
@pytest.mark.parametrize("cap,budget,recent", [(40, 16, 5), (700, 300, 64), (700, 1, 0), (300, 299, 299)])
def test_eviction_of_many_rows(in_place, kind, cap, budget, recent):
    layers, Bn, KV = 20, -(-2 * sms() // 160), 8
    many(layers, Bn, KV, cap)
    lens = [cap - (cap // 3) * b for b in range(Bn)]
    ops.run_evict(layers, KV, 16, "bf16", [max(n, 0) for n in lens], cap, budget, recent, in_place, kind=kind)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_eviction_of_many_long_rows(in_place, kind):
    # every register of a thread, and more slots to a thread than one word of bits
    cap, Bn = 8192, -(-2 * sms() // 32)
    many(32, Bn, 1, cap)
    lens = [8192, 8191, 4097] + [50 * b for b in range(Bn - 3)]
    ops.run_evict(32, 1, 16, "bf16", lens, cap, 1000, 33, in_place, kind=kind)


@pytest.mark.parametrize("in_place", [False, True])
def test_eviction_of_few_rows_by_registers_and_shared_keys(in_place):
    # 16384 slots are what 1024 threads hold in registers, 32768 what shared memory holds
    for n in (16384, 16385, 32768, 32769):
        ops.run_evict(1, 1, 16, "bf16", [n], n, 5000, 77, in_place, kind="ties")


@pytest.mark.parametrize("over", [1, 2, 7])
def test_eviction_of_a_few_slots_in_place(over):
    # a decode loop over its budget by the last step's tokens
    ops.run_evict(4, 8, 64, "bf16", [512 + over, 512, 511 + over], 520, 512, 128, True)
