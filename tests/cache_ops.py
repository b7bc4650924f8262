"""Shared set-up and 64-bit references for the tests of the read-back, the
window decode with sinks and the prefill attention."""
from __future__ import annotations

import numpy as np
import torch

import kvq_workloads as wl
from int8_quantized_paged_gb300 import kvq
from int8_quantized_paged_gb300.cache import LayerCache
from oracle import kvq_oracle as O

P = 16
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# layer shapes: a workload's, with some fields replaced
LAYERS = {
    "tiny": dict(name="tiny"),
    "tiny_f16": dict(name="tiny", act="f16"),
    "llama8b": dict(name="llama8b", n_heads=8, n_kv_heads=2),
    "llama8b_bf16": dict(name="llama8b", n_heads=8, n_kv_heads=2, act="bf16"),
    "g1": dict(name="llama8b", n_heads=2, n_kv_heads=2),
    "g2_int8": dict(name="llama8b", n_heads=4, n_kv_heads=2, k_kind="sym8", v_kind="sym8", k_group=64, v_group=64,
                    k_param="bf16", v_param="bf16"),
    "llama8b_f16": dict(name="llama8b_f16", n_heads=8, n_kv_heads=2, act="bf16"),
    "llama8b_shimmy": dict(name="llama8b_shimmy", n_heads=8, n_kv_heads=2),
    "long_mixed": dict(name="long_mixed", n_heads=16, n_kv_heads=2),
    "gemma": dict(name="gemma_mix", n_heads=4, n_kv_heads=2),
    "gemma_bf16": dict(name="gemma_mix", n_heads=4, n_kv_heads=2, act="bf16"),
    "int8_256": dict(name="gemma_mix", n_heads=4, n_kv_heads=2, k_kind="sym8", v_kind="sym4", k_group=32, v_group=32,
                     k_param="f16", v_param="f16"),
    "group16": dict(name="llama8b", n_heads=8, n_kv_heads=2, k_group=16, v_group=16),
    "mixed_groups": dict(name="llama8b", n_heads=8, n_kv_heads=2, k_group=32, v_group=128, k_param="f16"),
    "norope": dict(name="tiny", act="f16", rope="none"),
}


def layer(key: str, **over) -> dict:
    d = dict(LAYERS[key])
    return wl.workload(d.pop("name"), **{**d, **over})


def row_map(t, ring_rows: int, sinks: int):
    """Row of token t: append-only, or pinned pages for the sinks and a ring behind them."""
    t = np.asarray(t, np.int64)
    if not ring_rows:
        return t
    pin = -(-sinks // P) * P
    return np.where(t < pin, t, pin + (t - pin) % ring_rows)


class Cache:
    """A layer's cache filled token by token on the GPU, and its bytes on the CPU."""

    def __init__(self, w: dict, lens, sinks: int = 0, ring_rows: int = 0, extra_tokens: int = 0, seed: int = 0,
                 k_size: float = 1.0, v_size: float = 1.0):
        self.w, self.lens = w, [int(x) for x in lens]
        self.sinks, self.ring = sinks, ring_rows
        self.B = len(self.lens)
        self.cfg = kvq.config(**w)
        self.spec = O.Spec.from_workload({**w, "act": "f16"})
        self.act = TORCH[w["act"]]
        cap = max(self.lens) + extra_tokens
        rows = -(-sinks // P) * P + ring_rows if ring_rows else cap
        self.max_pages = max(1, -(-rows // P))
        n_pages = self.B * self.max_pages + 3
        pool = kvq.Pool(n_pages)
        pool.alloc(n_pages)
        pool.free(np.random.default_rng(seed + 1).permutation(n_pages).astype(np.int32))
        self.rope_max = max(2, cap + 1)
        self.c = LayerCache(self.cfg, self.B, self.max_pages, n_pages, self.rope_max, ring_rows, pool=pool,
                            sinks=sinks)
        # bytes no append has written look like anything: NaN scales, any code
        self.c.k_pool.fill_(0xFF)
        self.c.v_pool.fill_(0xFF)
        for b in range(self.B):
            self.c.reserve(b, rows if ring_rows else max(1, cap))
        self.c.sync_table()
        self.bt = self.c.table.data()
        self.gen = torch.Generator().manual_seed(seed)
        self.k_size, self.v_size = k_size, v_size
        step = ring_rows or (1 << 30)
        for b, L in enumerate(self.lens):
            for s in range(0, L, step):   # rows of one call never share a ring slot
                self.append(b, s, min(L, s + step))
        torch.cuda.synchronize()
        assert self.c.status_bits() == 0

    def rows(self, n: int, size: float = 1.0) -> torch.Tensor:
        x = torch.randn(n, self.w["n_kv_heads"], self.w["head_dim"], generator=self.gen)
        x = size * x
        if "f16" in (self.w["act"], self.w["k_kind"]):   # finite in fp16, rotated too
            x = x.clamp(-4e4, 4e4)
        return x.to(self.act).cuda()

    def append(self, b: int, s: int, e: int, k=None, v=None) -> None:
        k = self.rows(e - s, self.k_size) if k is None else k
        v = self.rows(e - s, self.v_size) if v is None else v
        self.c.append(k, v, torch.arange(s, e, dtype=torch.int32, device="cuda"),
                      torch.full((e - s,), b, dtype=torch.int32, device="cuda"))

    def queries(self, n: int, size: float = 1.0) -> torch.Tensor:
        if self.w["attn_scale"]:
            size /= 8.0   # a layer whose score scale is 1 has its queries normalised
        x = torch.randn(n, self.w["n_heads"], self.w["head_dim"], generator=self.gen)
        return (size * x).to(self.act).cuda()

    def pools(self):
        return {"k": self.c.k_pool.cpu().numpy(), "v": self.c.v_pool.cpu().numpy()}

    def values(self, pools, which: str, b: int, t) -> np.ndarray:
        """Stored rows of tokens t in 64 bits: [T][kv heads][head_dim]."""
        return O.gather_dequant(self.spec, which, pools[which], self.bt[b], row_map(t, self.ring, self.sinks))

    def rotated(self, q: torch.Tensor, pos) -> np.ndarray:
        """Queries [n][heads][head_dim] rotated at positions pos, in 64 bits."""
        s = self.spec
        x = q.double().cpu().numpy()
        return np.stack([O.rotate_f64(x[i], int(p), s.head_dim, s.rope_base, s.rope) for i, p in enumerate(pos)])

    def attend(self, pools, q: torch.Tensor, b: int, pos, window: int, sinks: int, left_out=()):
        """(out, score size) in 64 bits of queries at positions pos of sequence b: the largest
        alpha * sum_d |q_d k_d| of a row bounds how far rounded operands move its scores."""
        s = self.spec
        n, G, pos = len(pos), s.group_size, np.asarray(pos)
        out = np.zeros((n, s.n_heads, s.head_dim))
        size = np.zeros((n, s.n_heads))
        if not n:
            return out, size
        hi, lo = int(pos.max()) + 1, 0
        t = np.arange(hi)
        if window:
            lo = max(0, int(pos.min()) - window + 1)
            t = t[(t >= lo) | (t < sinks)]
        t = t[~np.isin(t, left_out)]
        see = t[None] <= pos[:, None]
        if window:
            see &= (t[None] > pos[:, None] - window) | (t[None] < sinks)
        K, V = self.values(pools, "k", b, t), self.values(pools, "v", b, t)
        x = self.rotated(q, pos)
        for h in range(s.n_heads):
            sc = np.where(see, s.alpha() * (x[:, h] @ K[:, h // G].T), -np.inf)
            m = np.max(sc, axis=1, keepdims=True, initial=-1e300)
            p = np.exp(sc - m)
            den = p.sum(1, keepdims=True)
            out[:, h] = (p / np.where(den == 0, 1, den)) @ np.where(np.isfinite(V[:, h // G]), V[:, h // G], 0)
            size[:, h] = np.max(np.where(see, s.alpha() * (np.abs(x[:, h]) @ np.abs(K[:, h // G]).T), 0), axis=1,
                                initial=0)
        return out, size

    def close(self):
        self.c.close()
