"""Host checks of kvq_read, the sink entry points and kvq_prefill_attention: refusals come
before any launch, so they run without a GPU."""
import ctypes as C

import pytest
import torch

import kvq_workloads as wl
from int8_quantized_paged_gb300 import kvq


def _cfg(**over):
    return kvq.config(**wl.workload("llama8b", **over))


BUF = torch.zeros(4096 + 256, dtype=torch.uint8)       # host memory: never dereferenced
A = (BUF.data_ptr() + 255) // 256 * 256                # aligned


def _read(cfg=None, n=2, ids=A, pos=A, table=A, n_seqs=2, pages=8, ring=0, sinks=0, kp=A, vp=A, n_pool=4, ko=A, vo=A,
          st=A):
    return kvq.lib().kvq_read(C.byref(cfg or _cfg()), n, ids, pos, table, n_seqs, pages, ring, sinks, kp, vp, n_pool,
                              ko, vo, st, None)


def _sink(cfg=None, B=2, q=A, kp=A, vp=A, n_pool=4, table=A, pages=64, ring=0, sinks=4, window=64, lens=A, rope=A,
          rmax=8, out=A, ws=A, wb=1 << 30, chunk=0, st=A):
    return kvq.lib().kvq_sink_decode(C.byref(cfg or _cfg()), B, q, kp, vp, n_pool, table, pages, ring, sinks, window,
                                     lens, rope, rmax, out, ws, wb, chunk, st, None)


def _fused(cfg=None, B=2, q=A, k=A, v=A, pos=A, kp=A, vp=A, n_pool=4, table=A, pages=64, ring=0, sinks=4, window=64,
           lens=A, rope=A, rmax=8, out=A, ws=A, wb=1 << 30, chunk=0, st=A):
    return kvq.lib().kvq_append_sink_decode(C.byref(cfg or _cfg()), B, q, k, v, pos, kp, vp, n_pool, table, pages,
                                            ring, sinks, window, lens, rope, rmax, out, ws, wb, chunk, st, None)


def _append(cfg=None, n=2, k=A, v=A, ids=A, pos=A, table=A, n_seqs=2, pages=8, ring=0, sinks=0, rope=A, rmax=8, kp=A,
            vp=A, n_pool=4, st=A):
    return kvq.lib().kvq_append_sink(C.byref(cfg or _cfg()), n, k, v, ids, pos, table, n_seqs, pages, ring, sinks,
                                     rope, rmax, kp, vp, n_pool, st, None)


def _prefill(cfg=None, B=2, n=10, q=A, starts=A, kp=A, vp=A, n_pool=4, table=A, pages=64, ring=0, sinks=0, window=0,
             lens=A, rope=A, rmax=8, out=A, ws=A, wb=1 << 30, st=A):
    return kvq.lib().kvq_prefill_attention(C.byref(cfg or _cfg()), B, n, q, starts, kp, vp, n_pool, table, pages, ring,
                                           sinks, window, lens, rope, rmax, out, ws, wb, st, None)


INV, SMALL, UNS = kvq.ERR_INVALID_ARG, kvq.ERR_WORKSPACE_TOO_SMALL, kvq.ERR_UNSUPPORTED


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), INV), (dict(pos=None), INV), (dict(table=None), INV), (dict(st=None), INV),
    (dict(ko=None, vo=None), INV), (dict(kp=None), INV), (dict(vp=None), INV), (dict(n_seqs=0), INV),
    (dict(pages=0), INV), (dict(n_pool=0), INV), (dict(ids=None, n=3), INV), (dict(ring=20), INV),
    (dict(ring=-16), INV), (dict(ring=16 * 9), INV), (dict(ring=16 * 8, sinks=1), INV), (dict(sinks=-1), INV),
    (dict(kp=A + 8), INV), (dict(ko=A + 2), INV), (dict(vo=A + 8), INV), (dict(cfg=_cfg(head_dim=96)), INV),
])
def test_read_refuses(over, want):
    assert _read(**over) == want
    assert kvq.last_error()


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), INV), (dict(k=None), INV), (dict(ring=16 * 8, sinks=1), INV), (dict(sinks=-1), INV),
    (dict(rope=None), INV), (dict(kp=A + 8), INV), (dict(ids=None, n=3), INV),
])
def test_append_sink_refuses(over, want):
    assert _append(**over) == want


SINK = [
    (dict(B=-1), INV), (dict(q=None), INV), (dict(lens=None), INV), (dict(out=None), INV), (dict(ws=None), INV),
    (dict(window=0), INV), (dict(window=-3), INV), (dict(sinks=-1), INV), (dict(ring=32, window=33), INV),
    (dict(ring=16 * 64, window=5), INV), (dict(ring=24), INV), (dict(pages=0), INV), (dict(chunk=8), INV),
    (dict(chunk=-16), INV), (dict(wb=64), SMALL), (dict(q=A + 8), INV), (dict(ws=A + 16), INV), (dict(rope=None), INV),
    (dict(cfg=_cfg(n_heads=48, n_kv_heads=3)), UNS),
]


@pytest.mark.parametrize("over,want", SINK)
def test_sink_decode_refuses(over, want):
    assert _sink(**over) == want


@pytest.mark.parametrize("over,want", SINK + [(dict(k=None), INV), (dict(pos=None), INV), (dict(v=A + 8), INV),
                                              (dict(cfg=_cfg(k_group=16, v_group=16), wb=64), SMALL)])
def test_append_sink_decode_refuses(over, want):
    assert _fused(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(B=-1), INV), (dict(n=-1), INV), (dict(q=None), INV), (dict(starts=None), INV), (dict(lens=None), INV),
    (dict(out=None), INV), (dict(ws=None), INV), (dict(st=None), INV), (dict(window=-1), INV), (dict(sinks=-1), INV),
    (dict(sinks=4), INV), (dict(ring=32), INV), (dict(ring=32, window=33), INV), (dict(ring=24, window=5), INV),
    (dict(ring=16 * 64, window=5, sinks=1), INV), (dict(pages=0), INV), (dict(n_pool=0), INV), (dict(wb=8), SMALL),
    (dict(q=A + 8), INV), (dict(out=A + 8), INV), (dict(ws=A + 16), INV), (dict(kp=A + 8), INV),
    (dict(rope=A + 8), INV), (dict(rope=None), INV), (dict(rmax=0), INV), (dict(cfg=_cfg(page_size=32)), UNS),
])
def test_prefill_refuses(over, want):
    assert _prefill(**over) == want


def test_nothing_to_do_is_fine():
    assert _read(n=0) == _append(n=0) == _sink(B=0) == _fused(B=0) == kvq.OK
    assert _prefill(B=0) == _prefill(n=0) == kvq.OK


@pytest.mark.parametrize("call", [_read, _append, _sink, _fused, _prefill])
def test_unknown_flags_and_no_config(call):
    c = _cfg()
    c.flags = 1 << 4
    assert call(cfg=c) == INV and "flags" in kvq.last_error()


def test_workspace_sizes():
    c = _cfg()
    # a window is far smaller than the context it slides over, and sinks add their pages
    small = kvq.sink_workspace_bytes(c, 4, 2048, 0, 4, 1024, 64)
    assert small < kvq.decode_workspace_bytes(c, 4, 2048, 64)
    assert kvq.sink_workspace_bytes(c, 4, 2048, 0, 4096, 1024, 64) > small
    # the whole context in sight: no more than the context needs, and a block for the window's start
    assert kvq.sink_workspace_bytes(c, 4, 64, 0, 1 << 30, 1 << 30, 64) <= \
        kvq.decode_workspace_bytes(c, 4, 65, 64) + 4096
    # prefill: nothing but a pad when the tiles fill the GPU; parts of the keys when they do not
    assert kvq.prefill_workspace_bytes(c, 1, 8192, 512) < 4096
    few = kvq.prefill_workspace_bytes(c, 1, 5, 512)
    assert few > 5 * 32 * 128 * 4
    for bad in (dict(batch=-1), dict(n_rows=-1), dict(max_pages_per_seq=0), dict(ring_rows=24, window=8),
                dict(sinks=3), dict(window=-1)):
        a = {**dict(batch=1, n_rows=4, max_pages_per_seq=8, ring_rows=0, sinks=0, window=0), **bad}
        with pytest.raises(kvq.KvqError):
            kvq.prefill_workspace_bytes(c, **a)
    for bad in (dict(window=0), dict(sinks=-1), dict(ring_rows=16, window=17), dict(chunk_tokens=5)):
        a = {**dict(batch=1, max_pages_per_seq=8, ring_rows=0, sinks=0, window=8, chunk_tokens=0), **bad}
        with pytest.raises(kvq.KvqError):
            kvq.sink_workspace_bytes(c, **a)


def test_layer_cache_refusals():
    """Calls whose tensors or layout do not fit are refused before anything is launched."""
    from int8_quantized_paged_gb300.cache import LayerCache
    c = LayerCache(_cfg(), 1, 8, 8, rope_max_pos=64, ring_rows=32, device="cpu", sinks=4)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)   # noqa: E731
    rows = lambda n, h=32, t=torch.float16: torch.zeros(n, h, 128, dtype=t)   # noqa: E731
    ws = torch.zeros(64, dtype=torch.uint8)
    # a ring behind pinned pages is not the ring that the plain window decode reads
    with pytest.raises(ValueError, match="sink_decode"):
        c.window_decode(rows(1), i32(1), rows(1), ws, 16)
    with pytest.raises(ValueError, match="sink_decode"):
        c.append_window_decode(rows(1), rows(1, 8), rows(1, 8), i32(1), i32(1), rows(1), ws, 16)
    for k, v in ((rows(2, 8), rows(3, 8)), (rows(3, 8, torch.float32), None), (rows(3, 4), None)):
        with pytest.raises(ValueError, match="tensor is"):
            c.read(i32(3), k_out=k, v_out=v)
    for q, out in ((rows(3), rows(2)), (rows(3), rows(3, t=torch.bfloat16)), (rows(3, 8), rows(3, 8))):
        with pytest.raises(ValueError, match="tensor is"):
            c.prefill(q, i32(2), i32(1), out, ws, 16)
    with pytest.raises(ValueError, match="q_starts"):
        c.prefill(rows(3), i32(3), i32(1), rows(3), ws, 16)
    c.close()
