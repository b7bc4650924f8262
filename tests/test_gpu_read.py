"""kvq_read: stored rows back as numbers, against the oracle's 64-bit values.

A stored value is s * code (+ bias): one fp32 rounding (2^-24 of the value; with a
bias the fused multiply-add rounds the sum once), then one rounding to the
activation type (half a step, eps / 2).  Both are relative to the result, so the
bound is (2^-24 + eps / 2) |value|, plus half the smallest subnormal step of fp16.
"""
import numpy as np
import pytest
import torch

from cache_ops import LAYERS, TORCH, Cache, layer
from int8_quantized_paged_gb300 import kvq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    torch.cuda.init()


def _near(got: torch.Tensor, ref: np.ndarray, act: str):
    half = torch.finfo(TORCH[act]).eps / 2
    tiny = 2.0 ** -25 if act == "f16" else 0.0
    got = got.double().cpu().numpy()
    bound = (2.0 ** -24 + half) * (1 + 2.0 ** -10) * np.abs(ref) + tiny
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("key", list(LAYERS))
@pytest.mark.parametrize("act", ["f32", "f16", "bf16"])
def test_rows_match_the_stored_values(key, act):
    lens = [1, 37, 250]
    c = Cache(layer(key, act=act), lens)
    pools = c.pools()
    # every row of every sequence, in a shuffled order, one of them three times
    ids = np.concatenate([np.full(L, b) for b, L in enumerate(lens)] + [[1, 1]]).astype(np.int32)
    pos = np.concatenate([np.arange(L) for L in lens] + [[5, 5]]).astype(np.int32)
    order = np.random.default_rng(3).permutation(len(ids))
    ids, pos = ids[order], pos[order]
    k, v = c.c.read(torch.from_numpy(pos).cuda(), torch.from_numpy(ids).cuda())
    torch.cuda.synchronize()
    assert c.c.status_bits() == 0
    for b in range(len(lens)):
        at = np.nonzero(ids == b)[0]
        _near(k[at], c.values(pools, "k", b, pos[at]), act)
        _near(v[at], c.values(pools, "v", b, pos[at]), act)
    c.close()


@pytest.mark.parametrize("sinks,ring", [(0, 48), (4, 48), (17, 32)])
def test_ring_with_pinned_pages(sinks, ring):
    L = 203
    c = Cache(layer("gemma"), [L, 9], sinks=sinks, ring_rows=ring)
    pools = c.pools()
    pin = -(-sinks // 16) * 16
    t = np.concatenate([np.arange(pin), np.arange(L - ring, L)]).astype(np.int32)
    k, v = c.c.read(torch.from_numpy(t).cuda(), torch.zeros(len(t), dtype=torch.int32, device="cuda"))
    _near(k, c.values(pools, "k", 0, t), "f16")
    _near(v, c.values(pools, "v", 0, t), "f16")
    c.close()


def test_append_sink_writes_the_rows_kvq_append_writes():
    """A pinned ring holds, for every token it still has, the bytes that an append-only cache holds."""
    w = layer("long_mixed")
    L, sinks, ring = 170, 20, 64
    a = Cache(w, [L])
    b = Cache(w, [L], sinks=sinks, ring_rows=ring)
    t = np.concatenate([np.arange(32), np.arange(L - ring, L)]).astype(np.int32)
    k = a.rows(L)
    v = a.rows(L)
    a.append(0, 0, L, k, v)
    for s in range(0, L, ring):
        e = min(L, s + ring)
        b.append(0, s, e, k[s:e].contiguous(), v[s:e].contiguous())
    tt = torch.from_numpy(t).cuda()
    zero = torch.zeros(len(t), dtype=torch.int32, device="cuda")
    for x, y in zip(a.c.read(tt, zero), b.c.read(tt, zero)):
        assert torch.equal(x, y)
    assert b.c.status_bits() == 0
    a.close()
    b.close()


def test_one_output_only_and_no_sequence_ids():
    c = Cache(layer("llama8b"), [20, 30, 40])
    pos = torch.tensor([3, 29, 39], dtype=torch.int32, device="cuda")   # row i of sequence i
    k, v = c.c.read(pos)
    ids = torch.arange(3, dtype=torch.int32, device="cuda")
    k2 = torch.full_like(k, 7)
    kvq.read(c.cfg, ids, pos, c.c.block_table, 3, c.max_pages, 0, 0, c.c.k_pool, None, c.c.n_pool_pages, k2, None,
             c.c.status)
    assert torch.equal(k, k2)
    v2 = torch.full_like(v, 7)
    kvq.read(c.cfg, ids, pos, c.c.block_table, 3, c.max_pages, 0, 0, None, c.c.v_pool, c.c.n_pool_pages, None, v2,
             c.c.status)
    assert torch.equal(v, v2)
    c.close()


def test_bad_rows_are_flagged_and_left_as_they_were():
    c = Cache(layer("llama8b"), [20, 30])
    c.c.block_table[1, 1] = c.c.n_pool_pages          # a page outside the pool
    pos = torch.tensor([3, -1, 32, 3, 17, 5], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 0, 0, 2, 1, 1], dtype=torch.int32, device="cuda")
    k = torch.full((6, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    v = k.clone()
    c.c.read(pos, ids, k, v)
    assert c.c.status_bits() == kvq.DEV_BAD_POS | kvq.DEV_BAD_SEQ | kvq.DEV_BAD_PAGE
    for i in (1, 2, 3, 4):
        assert torch.all(k[i] == 7) and torch.all(v[i] == 7)
    for i in (0, 5):
        assert not torch.all(k[i] == 7) and not torch.all(v[i] == 7)
    c.close()


def test_captured_into_a_graph_on_a_side_stream():
    c = Cache(layer("long_mixed"), [100])
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    ids = torch.zeros(100, dtype=torch.int32, device="cuda")
    want = c.c.read(pos, ids)
    out = tuple(torch.zeros_like(x) for x in want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.c.read(pos, ids, *out)
    for _ in range(2):
        for x in out:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    c.close()
