"""kvq_prefill_attention on the GPU against a 64-bit reference over the pool's own bytes.

Bounds.  Let u be half a step of the operands (2^-11 where the products run on the
tensor cores in fp16, 2^-24 in the fp32 kernel).  A rotated query carries one rounding, a
stored value at most two (its scale and the product): a score is off by at most
D = size * (3 u + (hd + 8) 2^-24), size = max_t alpha sum_d |q_d k_td|, the second term the
fp32 sum.  Softmax weights change by a factor within e^(+-2D), a weight and a value carry
three more roundings and the sum over T keys T 2^-24, so
  |out - ref| <= ((e^(2D) - 1) + 1.05 (3 u + (T + 16) 2^-24)) max|V| + half |ref|,
half = eps / 2 of the activation type.  That is a worst case; roundings are independent, so
the 2-norm of the error is held to 4 u (1 + s) + half of the result's, s the spread of the
scores (about 1, and 2 for the layer with score scale 1): six roundings of rms u / sqrt(3)
make 1.4 u s, and the fp32 kernel's sums of hd terms are covered by u * sqrt(hd).
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


def _starts(news, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(news)]), dtype=torch.int32, device="cuda")


def _prefill(c: Cache, q, news, window: int = 0, lens=None, first: int = 0, stream=None):
    lens = torch.tensor(c.lens if lens is None else lens, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = c.c.prefill_workspace(c.B, len(q), window)
    ws.fill_(0xFF)                                     # it needs no clearing
    c.c.prefill(q, _starts(news, first), lens, out, ws, window, stream=stream)
    torch.cuda.synchronize()
    return out


def _half_precision(w):
    return w["act"] != "f32" and (w["k_kind"] == "f16" or min(w["k_group"], w["v_group"]) >= 32)


def _near(c: Cache, pools, got, q, b, pos, window, norm=True, left_out=()):
    sinks = c.sinks if window else 0
    ref, size = c.attend(pools, q, b, pos, window, sinks, left_out)
    got = got.double().cpu().numpy()
    T, hd = int(max(pos)) + 1, c.w["head_dim"]
    u = 2.0 ** -11 if _half_precision(c.w) else 2.0 ** -24
    half = torch.finfo(TORCH[c.w["act"]]).eps / 2
    V = c.values(pools, "v", b, np.arange(T) if not c.ring else
                 np.arange(max(0, T - c.ring), T))
    big = np.max(np.abs(V[np.isfinite(V)]))
    D = size * (3 * u + (hd + 8) * 2.0 ** -24)
    bound = (np.expm1(2 * D) + 1.05 * (3 * u + (T + 16) * 2.0 ** -24)) * big
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got))
    assert np.all(err <= bound[..., None] + half * np.abs(ref) + 2.0 ** -25), float(err.max())
    if norm:
        s = 2.0 if c.w["attn_scale"] else 1.0
        tol = 4 * u * (1 + s) * (1 if _half_precision(c.w) else hd ** 0.5) + half
        rel = np.linalg.norm(err) / np.linalg.norm(ref)
        assert rel <= tol, (rel, tol)


def _check(c: Cache, q, out, news, window: int = 0, lens=None, first: int = 0, **kw):
    pools, at = c.pools(), first
    for b, (n, L) in enumerate(zip(news, c.lens if lens is None else lens)):
        if n:
            _near(c, pools, out[at:at + n], q[at:at + n], b, np.arange(L - n, L), window, **kw)
        at += n


LENS, NEWS = [1, 5, 17, 300, 33, 513], [1, 5, 0, 64, 33, 100]


@pytest.mark.parametrize("key", list(LAYERS))
@pytest.mark.parametrize("sinks,window", [(0, 0), (4, 50), (17, 16), (0, 1), (3, 1000), (200, 40)])
def test_ragged_batch(key, sinks, window):
    c = Cache(layer(key), LENS, sinks=sinks)
    q = c.queries(sum(NEWS))
    out = _prefill(c, q, NEWS, window)
    assert c.c.status_bits() == 0
    _check(c, q, out, NEWS, window)
    c.close()


@pytest.mark.parametrize("key", ["tiny", "tiny_f16", "llama8b", "llama8b_bf16", "llama8b_f16", "g1", "long_mixed",
                                 "gemma", "int8_256"])
@pytest.mark.parametrize("n,L", [(600, 1500), (1, 2500), (257, 257), (128, 4097), (7, 6000)])
def test_one_sequence(key, n, L):
    c = Cache(layer(key), [L])
    q = c.queries(n)
    out = _prefill(c, q, [n])
    assert c.c.status_bits() == 0
    _check(c, q, out, [n])
    c.close()


@pytest.mark.parametrize("key", ["tiny", "llama8b", "llama8b_bf16", "long_mixed", "gemma", "llama8b_f16", "group16"])
@pytest.mark.parametrize("sinks,window,ring", [(4, 50, 96), (0, 33, 96), (33, 100, 112)])
def test_chunk_through_a_ring(key, sinks, window, ring):
    n = ring - window + 1                              # the longest chunk the ring allows
    lens, news = [400, n, 100, 13], [n, n, 1, 13 if n >= 13 else n]
    c = Cache(layer(key), lens, sinks=sinks, ring_rows=ring)
    q = c.queries(sum(news))
    out = _prefill(c, q, news, window)
    assert c.c.status_bits() == 0
    _check(c, q, out, news, window)
    c.close()


def test_long_window_tiles():
    """Windows and sinks that cross key tiles, far into the context."""
    for key in ("llama8b", "gemma", "tiny_f16", "tiny"):
        for sinks, window in ((4, 300), (150, 129), (128, 700)):
            c = Cache(layer(key), [1700], sinks=sinks)
            q = c.queries(500)
            _check(c, q, _prefill(c, q, [500], window), [500], window)
            c.close()


def test_rows_of_no_sequence_are_left_as_they_were():
    for key in ("llama8b", "tiny"):
        c = Cache(layer(key), [40, 100])
        q = c.queries(3 + 30 + 20 + 9)
        out = _prefill(c, q, [30, 20], first=3)
        assert c.c.status_bits() == 0
        assert torch.all(out[:3] == 7) and torch.all(out[53:] == 7)
        _check(c, q, out, [30, 20], first=3)
        c.close()


def test_single_token_agrees_with_decode():
    c = Cache(layer("llama8b"), [700, 33])
    q = c.queries(2)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    dec = torch.full_like(q, float("nan"))
    c.c.decode(q, lens, dec, c.c.workspace(2))
    out = _prefill(c, q, [1, 1])
    rel = (out.double() - dec.double()).norm() / dec.double().norm()
    assert rel <= 8 * 2.0 ** -11 + 2.0 ** -11
    c.close()


@pytest.mark.parametrize("key,k_size,v_size", [
    ("llama8b", 3e4, 3e4), ("llama8b", 1e-3, 1e-3), ("llama8b_bf16", 1e30, 1e30), ("llama8b_bf16", 1e-20, 1e-20),
    ("gemma_bf16", 1e10, 1e-10), ("llama8b_f16", 2e4, 2e-3)])
def test_ranges(key, k_size, v_size):
    """Keys and values far from 1: operands are held at a power-of-two scale of their own."""
    c = Cache(layer(key), [400, 90], k_size=k_size, v_size=v_size)
    q = c.queries(150 + 90, size=1.0 / k_size)
    if key == "llama8b_f16":                           # stored rows are fp16
        assert torch.isfinite(c.rows(8, k_size)).all()
    out = _prefill(c, q, [150, 90])
    assert c.c.status_bits() == 0
    pools, at = c.pools(), 0
    for b, n in enumerate([150, 90]):
        L = c.lens[b]
        ref, _ = c.attend(pools, q[at:at + n], b, np.arange(L - n, L), 0, 0)
        got = out[at:at + n].double().cpu().numpy()
        half = torch.finfo(c.act).eps / 2
        # scores of about N(0, 1) (2 with score scale 1) as in the other tests.  fp16 queries of 1 / 3e4
        # are subnormal, exact as inputs; fp16 results of 1e-3 and less round at 2^-25
        tiny = 2.0 ** -25 * ref.size ** 0.5 if c.w["act"] == "f16" else 0.0
        s = 2.0 if c.w["attn_scale"] else 1.0
        tol = (4 * 2.0 ** -11 * (1 + s) + half) * np.linalg.norm(ref) + tiny
        assert np.linalg.norm(got - ref) <= tol, np.linalg.norm(got - ref) / np.linalg.norm(ref)
        at += n
    c.close()


@pytest.mark.parametrize("key", ["llama8b", "llama8b_shimmy", "tiny_f16", "int8_256", "gemma"])
@pytest.mark.parametrize("below", [0, 1, 2, 4, 8, 16])
def test_scales_just_below_a_power_of_two(key, below):
    """The largest scale of a step may round up to the next power of two in fp16."""
    c = Cache(layer(key), [400])
    s = c.spec
    for which, pool in (("k", c.c.k_pool), ("v", c.c.v_pool)):
        kind, group, param = ((s.k_kind, s.k_group, s.k_param) if which == "k" else (s.v_kind, s.v_group, s.v_param))
        cb = s.head_dim * (8 if kind == "sym8" else 4) // 8
        pb = s.head_dim // group * (2 if kind == "affine4" else 1) * (4 if param == "f32" else 2)
        par = pool.view(-1, s.n_kv_heads, 16 * (cb + pb))[:, :, 16 * cb:]
        x = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[param]
        v = torch.nextafter(torch.tensor(2.0), torch.tensor(0.0)) if below == 0 else torch.tensor(2.0 - below * 2.0 ** -13)
        vals = par.contiguous().view(x)
        vals[..., ::2 if kind == "affine4" else 1] = v.to(x).cuda()   # the scales, not the biases
        par.copy_(vals.view(torch.uint8))
    q = c.queries(300, size=0.25)
    out = _prefill(c, q, [300])
    assert c.c.status_bits() == 0
    _check(c, q, out, [300], norm=False)
    c.close()


@pytest.mark.parametrize("key", ["llama8b_bf16", "gemma", "llama8b_f16", "tiny"])
@pytest.mark.parametrize("grow", [True, False])
def test_values_that_grow_or_shrink_along_the_context(key, grow):
    L = 900
    c = Cache(layer(key), [L])
    e = torch.linspace(-3, 3, L) if grow else torch.linspace(3, -3, L)
    f = (10.0 ** e)[:, None, None].cuda()
    k = c.rows(L)
    v = (c.rows(L).float() * f).to(c.act)
    c.append(0, 0, L, k, v)
    q = c.queries(300)
    _check(c, q, _prefill(c, q, [300]), [300], norm=False)
    c.close()


@pytest.mark.parametrize("key", ["llama8b", "llama8b_bf16", "llama8b_f16", "gemma", "long_mixed", "tiny"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_token_that_is_not_finite_reaches_only_rows_that_attend_it(key, which):
    L, n, bad, window = 400, 250, 260, 60
    for w in (0, window):
        c = Cache(layer(key), [L])
        q = c.queries(n)
        clean = _prefill(c, q, [n], w)
        x, y = c.rows(1), c.rows(1)
        (x if which == "k" else y)[0, 0, 5] = float("inf")      # kv head 0 only
        c.append(0, bad, bad + 1, x, y)
        out = _prefill(c, q, [n], w)
        G = c.spec.group_size
        pos = np.arange(L - n, L)
        hit = (pos >= bad) & ((pos < bad + w) if w else True)
        got = out.float().cpu().numpy()
        assert np.all(np.isnan(got[hit][:, :G]))
        assert np.all(np.isfinite(got[~hit])) and np.all(np.isfinite(got[:, G:]))
        before = torch.from_numpy(pos < bad).cuda()
        assert torch.equal(out[before], clean[before])
        c.close()


def test_masked_rows_of_a_page_may_hold_anything():
    """Unwritten rows behind the last token hold NaN scales (the pools are filled with 0xFF), and
    tokens between the sinks and the window are not looked at."""
    for key in ("llama8b", "gemma", "llama8b_f16", "tiny"):
        c = Cache(layer(key), [500], sinks=4)
        q = c.queries(40)
        want = _prefill(c, q, [40], 60)
        junk = torch.full((300, c.w["n_kv_heads"], c.w["head_dim"]), float("inf"), device="cuda").to(c.act)
        c.append(0, 4, 304, junk, junk)
        got = _prefill(c, q, [40], 60)
        assert torch.all(torch.isfinite(got.float()))
        rel = (got.double() - want.double()).norm() / want.double().norm()
        assert rel <= 2.0 ** -9                         # the tiles may be grouped as before, or not
        c.close()


def test_a_query_that_is_not_finite_spoils_its_own_rows_only():
    c = Cache(layer("llama8b"), [300])
    q = c.queries(200)
    clean = _prefill(c, q, [200])
    q2 = q.clone()
    q2[77, 3, 9] = float("inf")
    out = _prefill(c, q2, [200])
    keep = torch.ones(200, 8, dtype=torch.bool, device="cuda")
    keep[77, 3] = False
    assert torch.equal(out[keep], clean[keep])
    assert torch.isnan(out[77, 3]).all()
    c.close()


@pytest.mark.parametrize("key", ["llama8b", "tiny"])
def test_bad_input_is_flagged(key):
    c = Cache(layer(key), [100, 64, 80, 200])
    news = [10, 64, 20, 30]
    q = c.queries(sum(news))
    hd = c.w["head_dim"]
    pools = c.pools()
    cases = [([100, 10 ** 6, 80, 200], kvq.DEV_BAD_LEN), ([100, 63, 80, 200], kvq.DEV_BAD_LEN),
             ([100, -1, 80, 200], kvq.DEV_BAD_LEN)]
    for lens, bit in cases:
        out = _prefill(c, q, news, lens=lens)
        assert c.c.status_bits() == bit
        kvq.clear_device_status(c.c.status)
        assert not out[10:74].any()                    # zero rows
        for b, (at, n) in enumerate([(0, 10), (None, 0), (74, 20), (94, 30)]):
            if n:
                _near(c, pools, out[at:at + n], q[at:at + n], b, np.arange(c.lens[b] - n, c.lens[b]), 0)
    # starts out of order or outside the rows: those sequences are left out
    for starts in ([0, 10, 5, 94, 124], [0, 10, 74, 94, 5000], [-5, 10, 74, 94, 124]):
        out = torch.full_like(q, 7.0)
        ws = c.c.prefill_workspace(c.B, len(q))
        c.c.prefill(q, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                    torch.tensor(c.lens, dtype=torch.int32, device="cuda"), out, ws)
        torch.cuda.synchronize()
        assert c.c.status_bits() & kvq.DEV_BAD_SEQ
        assert c.c.status_bits() & ~(kvq.DEV_BAD_SEQ | kvq.DEV_BAD_LEN) == 0
        kvq.clear_device_status(c.c.status)
    # a page outside the pool: its tokens are left out
    c.c.block_table[3, 2] = c.c.n_pool_pages
    out = _prefill(c, q, news)
    assert c.c.status_bits() == kvq.DEV_BAD_PAGE
    kvq.clear_device_status(c.c.status)
    _near(c, pools, out[94:], q[94:], 3, np.arange(170, 200), 0, left_out=range(32, 48))
    # a RoPE table that ends before the last position
    c.c.rope_max_pos = 150
    out = _prefill(c, q, news)
    assert c.c.status_bits() == kvq.DEV_BAD_POS | kvq.DEV_BAD_PAGE or c.c.status_bits() == kvq.DEV_BAD_POS
    assert not out[94:].any() and hd
    c.close()


def test_ring_rows_already_overwritten_are_flagged():
    c = Cache(layer("llama8b"), [300, 60], sinks=4, ring_rows=96)
    q = c.queries(80)
    out = _prefill(c, q, [48, 32], 50)                 # 48 + 50 - 1 = 97 > 96
    assert c.c.status_bits() == kvq.DEV_BAD_LEN
    assert not out[:48].any()
    _near(c, c.pools(), out[48:], q[48:], 1, np.arange(28, 60), 50)
    c.close()


def test_pages_that_all_sequences_share():
    """The same pages in two block-table rows (a shared prefix)."""
    c = Cache(layer("llama8b"), [128, 128])
    c.c.block_table[1] = c.c.block_table[0]
    c.bt[1] = c.bt[0]
    q = c.queries(100)
    q[50:] = q[:50]
    out = _prefill(c, q, [50, 50])
    assert torch.equal(out[:50], out[50:])
    _check(c, q, out, [50, 50])
    c.close()


def test_streams_and_graphs():
    c = Cache(layer("llama8b"), [900, 40])
    q = c.queries(60)
    want = _prefill(c, q, [40, 20])
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    st = _starts([40, 20])
    outs = [torch.zeros_like(q) for _ in range(2)]
    ws = [c.c.prefill_workspace(2, 60) for _ in range(2)]
    torch.cuda.synchronize()
    for i, s in enumerate((torch.cuda.Stream(), torch.cuda.Stream())):
        with torch.cuda.stream(s):
            for _ in range(4):
                c.c.prefill(q, st, lens, outs[i], ws[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # two captured graphs that share a workspace, replayed one after the other
    gs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.c.prefill(q, st, lens, outs[i], ws[0])
        gs.append(g)
    for _ in range(2):
        for o in outs:
            o.zero_()
        for g in gs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    c.close()


@pytest.mark.parametrize("key", ["llama8b", "llama8b_f16", "gemma", "tiny_f16"])
def test_calls_back_to_back(key):
    """Many calls with nothing between them: no wait inside the kernel runs out, and every call gives the same bits."""
    c = Cache(layer(key), [1500, 700, 64])
    news = [700, 699, 64]
    q = c.queries(sum(news))
    want = _prefill(c, q, news)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    st, out, ws = _starts(news), torch.empty_like(q), c.c.prefill_workspace(3, len(q))
    for _ in range(8):
        for _ in range(40):
            c.c.prefill(q, st, lens, out, ws)
        assert c.c.status_bits() == 0
        assert torch.equal(out, want)
    c.close()


@pytest.mark.parametrize("key", ["llama8b", "gemma_bf16", "tiny"])
def test_a_session(key):
    """As a server runs it: a prompt through a pinned ring in chunks, each appended and
    attended, then decode steps, then the window's rows read back."""
    sinks, window, ring = 4, 64, 96
    c = Cache(layer(key), [0, 0], sinks=sinks, ring_rows=ring, extra_tokens=400)
    lens = [0, 0]
    for n in (33, 20, 33, 1, 30):
        for b in range(2):
            c.append(b, lens[b], lens[b] + n)
        lens = [L + n for L in lens]
        q = c.queries(2 * n)
        out = _prefill(c, q, [n, n], window, lens=lens)
        _check(c, q, out, [n, n], window, lens=lens)
    ws = c.c.sink_workspace(2, window)
    for _ in range(20):
        lens = [L + 1 for L in lens]
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q, out = c.queries(2), None
        out = torch.empty_like(q)
        c.c.append_sink_decode(q, c.rows(2), c.rows(2), lt - 1, lt, out, ws, window)
    pre = _prefill(c, q, [1, 1], window, lens=lens)
    rel = (pre.double() - out.double()).norm() / out.double().norm()
    assert rel <= 3 * 4 * 2.0 ** -11 + torch.finfo(c.act).eps
    t = torch.arange(lens[0] - ring, lens[0], dtype=torch.int32, device="cuda")
    k, v = c.c.read(t, torch.zeros_like(t))
    pools = c.pools()
    for x, which in ((k, "k"), (v, "v")):
        ref = c.values(pools, which, 0, t.cpu().numpy())
        half = torch.finfo(c.act).eps / 2
        assert np.all(np.abs(x.double().cpu().numpy() - ref) <= (2.0 ** -23 + half) * np.abs(ref) + 2.0 ** -25)
    assert c.c.status_bits() == 0
    c.close()


@pytest.mark.parametrize("key", ["llama8b", "llama8b_bf16", "gemma", "gemma_bf16", "tiny_f16", "tiny", "g1"])
@pytest.mark.parametrize("n", [1, 2, 131])
def test_largest_queries(key, n):
    """Queries at fp16's upper end, which pass it when rotated, beside rows of zeros; a query that is
    not finite makes its own row NaN and no other."""
    top = 6.5e4
    w = layer(key)
    # scores of about N(0, 1) (2 with score scale 1), as in the other tests
    c = Cache(w, [max(n, 40) + 60], k_size=1.0 / top / (8.0 if w["attn_scale"] else 1.0))
    q = torch.sign(c.queries(n).float()).mul(top).to(c.act)
    q[1::3] = 0
    L = c.lens[0]
    out = _prefill(c, q, [n])
    assert c.c.status_bits() == 0
    pools = c.pools()
    _near(c, pools, out, q, 0, np.arange(L - n, L), 0)
    if n > 100:
        heads, hd = w["n_heads"], w["head_dim"]
        for i, x in ((5, "nan"), (6, "inf"), (77, "-inf")):
            q[i, i % heads, i % hd] = float(x)
        got = _prefill(c, q, [n])
        bad = torch.zeros(n, heads, dtype=torch.bool, device="cuda")
        for i in (5, 6, 77):
            bad[i, i % heads] = True
        assert torch.isnan(got[bad]).all()
        assert torch.equal(got[~bad], out[~bad])
    c.close()
