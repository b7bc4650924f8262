"""kvq_sink_decode, kvq_append_sink and kvq_append_sink_decode on the GPU, against
a 64-bit reference over the pool's own bytes, within the decode path's tolerance
(2e-3, row-relative with a 0.1 % floor, and normwise)."""
import numpy as np
import pytest
import torch

from cache_ops import Cache, layer
from gpu_cases import TOL, floor_for, max_row_err
from int8_quantized_paged_gb300 import kvq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    torch.cuda.init()


def _decode(c: Cache, q, window: int, lens=None, chunk: int = 0, stream=None):
    lens = torch.tensor(c.lens if lens is None else lens, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    c.c.sink_decode(q, lens, out, c.c.sink_workspace(len(q), window, chunk), window, chunk, stream=stream)
    torch.cuda.synchronize()
    return out


def _check(c: Cache, q, out, window: int, lens=None):
    pools = c.pools()
    act = c.w["act"]
    for b, L in enumerate(c.lens if lens is None else lens):
        got = out[b:b + 1].double().cpu().numpy()
        if L == 0:
            assert not got.any()
            continue
        ref, _ = c.attend(pools, q[b:b + 1], b, [L - 1], window, c.sinks)
        if act == "bf16":   # the result's own rounding: half a step is 2^-8
            assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + TOL * np.abs(ref).max(-1, keepdims=True))
        else:
            assert max_row_err(got, ref, floor=floor_for(c.w)) <= TOL, (b, L)


KEYS = ["tiny", "llama8b", "llama8b_bf16", "g1", "g2_int8", "llama8b_f16", "llama8b_shimmy", "long_mixed", "gemma",
        "group16", "mixed_groups", "norope"]


@pytest.mark.parametrize("key", KEYS)
@pytest.mark.parametrize("chunk", [0, 32])
@pytest.mark.parametrize("sinks,window", [(4, 50), (0, 33), (17, 16), (64, 100), (1, 1), (500, 20)])
def test_append_only_table(key, chunk, sinks, window):
    c = Cache(layer(key), [1, 16, 17, 70, 333, 0], sinks=sinks)
    q = c.queries(c.B)
    out = _decode(c, q, window, chunk=chunk)
    assert c.c.status_bits() == 0
    _check(c, q, out, window)
    c.close()


@pytest.mark.parametrize("key", ["tiny", "llama8b", "long_mixed", "gemma", "group16", "llama8b_f16"])
@pytest.mark.parametrize("sinks,window,ring", [(4, 50, 64), (0, 64, 64), (17, 16, 16), (33, 100, 112)])
def test_ring_behind_pinned_pages(key, sinks, window, ring):
    c = Cache(layer(key), [1, 16, 40, 333, 129], sinks=sinks, ring_rows=ring)
    q = c.queries(c.B)
    out = _decode(c, q, window)
    assert c.c.status_bits() == 0
    _check(c, q, out, window)
    c.close()


@pytest.mark.parametrize("key", ["tiny", "llama8b", "long_mixed", "gemma", "group16", "llama8b_shimmy"])
@pytest.mark.parametrize("ring", [0, 64])
def test_steps_of_the_fused_call(key, ring):
    """Token after token through append_sink_decode: the rows it writes are those of
    append_sink, and its output that of sink_decode on them, bit for bit."""
    w, sinks, window = layer(key), 5, 50
    a = Cache(w, [60, 3], sinks=sinks, ring_rows=ring, extra_tokens=40)
    b = Cache(w, [60, 3], sinks=sinks, ring_rows=ring, extra_tokens=40)
    ws = a.c.sink_workspace(2, window)
    for step in range(0, 40, 3):
        lens = [L + step + 1 for L in a.lens]
        k, v, q = a.rows(2), a.rows(2), a.queries(2)
        pos = torch.tensor(lens, dtype=torch.int32, device="cuda") - 1
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, float("nan"))
        a.c.append_sink_decode(q, k, v, pos, lt, out, ws, window)
        b.c.append(k, v, pos)
        want = _decode(b, q, window, lens)
        torch.cuda.synchronize()
        assert torch.equal(a.c.k_pool, b.c.k_pool) and torch.equal(a.c.v_pool, b.c.v_pool)
        assert torch.equal(out, want)
        if step % 9 == 0:
            _check(a, q, out, window, lens)
        for i in (1, 2):   # the two tokens between the steps
            if step + i < 40:
                k, v = a.rows(2), a.rows(2)
                for x in (a, b):
                    x.c.append(k, v, pos + i)
    assert a.c.status_bits() == 0 and b.c.status_bits() == 0
    a.close()
    b.close()


def test_window_past_the_context_is_plain_decode():
    c = Cache(layer("llama8b"), [200, 77], sinks=4)
    q = c.queries(2)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    want = torch.full_like(q, float("nan"))
    c.c.decode(q, lens, want, c.c.workspace(2, 64), 64)
    torch.cuda.synchronize()
    got = _decode(c, q, 100000, chunk=64)
    assert torch.equal(got, want)
    c.close()


def test_long_context_few_sinks():
    """A window far into a context, larger than one cluster: 4 sinks and 1500 tokens of 20000."""
    for key in ("llama8b", "gemma"):
        c = Cache(layer(key), [20000], sinks=4)
        q = c.queries(1)
        _check(c, q, _decode(c, q, 1500), 1500)
        c.close()


def test_masked_rows_of_a_page_may_hold_anything():
    """Tokens between the sinks and the window, and past the length, are not looked at."""
    c = Cache(layer("llama8b"), [100], sinks=4)
    q = c.queries(1)
    want = _decode(c, q, 20)
    big = torch.full((60, 2, 128), 60000.0, dtype=torch.float16, device="cuda")
    c.append(0, 10, 70, big, big)
    assert torch.equal(_decode(c, q, 20), want)
    c.close()


def test_bad_lengths_pages_and_positions():
    c = Cache(layer("llama8b"), [100, 100, 100], sinks=4)
    q = c.queries(3)
    c.c.block_table[2, 6] = -1                         # tokens 96 .. 99 left out
    out = _decode(c, q, 20, lens=[100, 100000, 100])
    bits = c.c.status_bits()
    assert bits == kvq.DEV_BAD_LEN | kvq.DEV_BAD_PAGE
    assert not out[1].any()
    pools = c.pools()
    ref, _ = c.attend(pools, q[2:3], 2, [99], 20, 4, left_out=range(96, 100))
    assert max_row_err(out[2:3].double().cpu().numpy(), ref) <= TOL
    kvq.clear_device_status(c.c.status)
    k = c.rows(3)
    before = c.c.k_pool.clone()
    c.c.append_sink_decode(q, k, k, torch.tensor([-1, 5000, 99], dtype=torch.int32, device="cuda"),
                           torch.tensor([100, 100, 50], dtype=torch.int32, device="cuda"), out,
                           c.c.sink_workspace(3, 20), 20)
    assert c.c.status_bits() == kvq.DEV_BAD_POS | kvq.DEV_BAD_PAGE
    assert torch.equal(c.c.k_pool, before)
    c.close()


def test_two_streams_and_a_graph():
    c = Cache(layer("llama8b"), [300, 40], sinks=20, ring_rows=64)
    q = c.queries(2)
    want = _decode(c, q, 60)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(2)]
    ws = [c.c.sink_workspace(2, 60) for _ in range(2)]     # calls that may overlap have their own
    torch.cuda.synchronize()
    for i, s in enumerate((torch.cuda.Stream(), torch.cuda.Stream())):
        with torch.cuda.stream(s):
            for _ in range(3):
                c.c.sink_decode(q, lens, outs[i], ws[i], 60)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.c.sink_decode(q, lens, outs[0], ws[0], 60)
    for _ in range(2):
        outs[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want)
    c.close()
