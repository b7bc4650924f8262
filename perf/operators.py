"""Cases and plain forms of the cache operators beside single-token decode.

Three operators of the quantised, paged KV cache:

* ``read``    -- rows of the cache back as numbers (kvq_read);
* ``sink``    -- one decode step of attention over a sliding window and a few first
                 tokens that stay visible (kvq_sink_decode);
* ``prefill`` -- causal attention of many new tokens per sequence over the cache, with
                 an optional window and first tokens (kvq_prefill_attention).

``run`` computes a case in elementary torch operations in 32 bits, or, where ``own`` is
true, with the library's calls.  The shapes are the ones of kvq_workloads.py and of the
tests: Llama-3.1-8B-shaped layers, the sliding + global mix, the long mixed-dtype context
and the tiny layer.
"""
import math
import random

import numpy as np
import torch

own = False

P = 16
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# The layers: query heads, kv heads, head_dim, K kind, V kind, group, stored scale type,
# score scale, RoPE pairing and base.
LAYERS = {
    "tiny": (4, 2, 64, "sym4", "sym4", 64, "f32", 0.0, "normal", 1e4),
    "llama8b": (32, 8, 128, "sym4", "sym4", 128, "f32", 0.0, "normal", 5e5),
    "llama8b_f16": (32, 8, 128, "f16", "f16", 128, "f32", 0.0, "normal", 5e5),
    "llama8b_shimmy": (32, 8, 128, "shimmy4", "shimmy4", 128, "f32", 0.0, "normal", 5e5),
    "long_mixed": (32, 4, 128, "sym8", "sym4", 32, "f16", 0.0, "normal", 5e5),
    "gemma_mix": (16, 8, 256, "affine4", "affine4", 64, "bf16", 1.0, "neox", 1e4),
}


def _case(name, op, layer, act, batch, new, ctx, ragged=False, window=0, sinks=0, ring=0):
    """new: query tokens (prefill) or rows read per sequence; ctx: tokens in the cache, the
    new ones included; ragged: both differ from sequence to sequence, up to these."""
    c = dict(op=op, layer=layer, act=act, batch=batch, new=new, ctx=ctx, ragged=ragged, window=window, sinks=sinks,
             ring=ring)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short shared prefix copied out of one sequence: latency
        _case("read_prefix", "read", "llama8b", "f16", 1, 37, 250),
        # a whole 16K sequence of the mix's global layer off-loaded as bf16
        _case("read_global_16k", "read", "gemma_mix", "bf16", 1, 16384, 16384),
        # every row of four 64K contexts, to be stored in another format
        _case("read_long_4x64k", "read", "long_mixed", "f16", 4, 65536, 65536),
        # the smallest layer, one token, fp32
        _case("sink_tiny", "sink", "tiny", "f32", 1, 1, 256, window=64, sinks=4),
        # the mix's window layer with four sinks beside its ring: one token of one user
        _case("sink_ring_16k", "sink", "gemma_mix", "f16", 1, 1, 16384, window=1024, sinks=4, ring=1152),
        # a continuous batch of streams that keep 4096 tokens and 64 first ones in sight
        _case("sink_batch_64", "sink", "llama8b", "f16", 64, 1, 32768, ragged=True, window=4096, sinks=64),
        # five drafted tokens checked at the end of an 8K context
        _case("prefill_verify_5", "prefill", "llama8b", "f16", 1, 5, 8192),
        # a short prompt on the smallest layer, fp32
        _case("prefill_tiny", "prefill", "tiny", "f32", 1, 100, 256),
        # a whole 8K prompt
        _case("prefill_prompt_8k", "prefill", "llama8b", "f16", 1, 8192, 8192),
        # a chunk of 2048 at the end of a 32K context of unquantised rows, bf16
        _case("prefill_chunk_32k", "prefill", "llama8b_f16", "bf16", 1, 2048, 32768),
        # the prompts of sixteen users in one call, each with its own history
        _case("prefill_ragged_16", "prefill", "llama8b_shimmy", "bf16", 16, 1024, 8192, ragged=True),
        # a prompt part through the mix's window layer with four sinks, head_dim 256
        _case("prefill_window_4k", "prefill", "gemma_mix", "f16", 1, 4096, 16384, window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    layer = rng.choice(list(LAYERS))
    act = "f32" if layer == "tiny" else rng.choice(("f16", "bf16"))
    op = rng.choice(("read", "sink", "prefill"))
    ragged = rng.random() < 0.5
    if op == "read":
        ctx = _log(rng, 16, 65536)
        batch = min(16, max(1, _log(rng, 1, 262144 / ctx)))
        return _case("", op, layer, act, batch, _log(rng, 1, ctx), ctx, ragged)
    window, sinks = _log(rng, 1, 8192), rng.choice((0, 1, 4, 16, 17, 64))
    if op == "sink":
        ring = (window + P - 1) // P * P + rng.choice((0, 16, 128)) if rng.random() < 0.5 else 0
        return _case("", op, layer, act, _log(rng, 1, 64), 1, _log(rng, 17, 32768), ragged, window, sinks, ring)
    if rng.random() < 0.6:
        window = sinks = 0
    ctx = _log(rng, 17, 8192 if layer == "tiny" else 32768)
    new = _log(rng, 1, min(ctx, 2048))
    # no more scores than the 8K prompt has
    most = max(1, min(16, 8192 * 8192 // (new * ctx)))
    # a chunk through a ring: the ring holds the first query's window and the chunk
    ring = (window + new + P - 2) // P * P + rng.choice((0, 16, 128)) if window and rng.random() < 0.5 else 0
    return _case("", op, layer, act, _log(rng, 1, most), new, ctx, ragged, window, sinks, ring)


def _lengths(case):
    """(new tokens, context) of every sequence: the case alone fixes them."""
    B, n, L = case["batch"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [n] * B, [L] * B
    r = random.Random("%d %d %d" % (B, n, L))
    lens = [r.randint(max(1, L // 64), L) for _ in range(B)]
    lens[r.randrange(B)] = L
    news = [min(k, r.randint(1, n)) for k in lens]
    return news, lens


# ---------------------------------------------------------------- inputs


def _bits(kind):
    return 16 if kind == "f16" else 8 if kind == "sym8" else 4


def _row_bytes(layer, which):
    """(code bytes, parameter bytes) of one token of one kv head."""
    hd, kind, group, param = layer[2], layer[3 + which], layer[5], layer[6]
    n = 0 if kind == "f16" else hd // group * (2 if kind == "affine4" else 1)
    return hd * _bits(kind) // 8, n * (4 if param == "f32" else 2)


def _stored(layer, which, x):
    """Rows x [pages, kv heads, 16, head_dim] (fp32) as pages of a pool."""
    hd, kind, group, pt = layer[2], layer[3 + which], layer[5], DT[layer[6]]
    lead = x.shape[:-1]
    if kind == "f16":
        codes, par = x.half().view(torch.uint8), None
    else:
        g = x.unflatten(-1, (hd // group, group))
        if kind == "affine4":
            lo = g.amin(-1, keepdim=True)
            s, b = ((g.amax(-1, keepdim=True) - lo) / 15).to(pt), lo.to(pt)
            q = torch.round((g - b.float()) / torch.where(s == 0, 1, s.float())).clamp(0, 15)
            par = torch.cat((s, b), -1)
        else:
            top = {"sym4": 7.0, "sym8": 127.0, "shimmy4": 7.5}[kind]
            s = (g.abs().amax(-1, keepdim=True) / top).clamp_min(2.0 ** -14).to(pt)
            low, high = (-8, 7) if kind == "shimmy4" else (-top, top)
            q = torch.round(g / s.float()).clamp(low, high) + (8 if kind == "shimmy4" else 0)
            par = s
        q = q.to(torch.int16).flatten(-2) & (255 if kind == "sym8" else 15)
        codes = (q if kind == "sym8" else q[..., 0::2] | q[..., 1::2] << 4).to(torch.uint8)
        par = par.contiguous().view(torch.uint8)
    codes = codes.reshape(*lead[:2], -1)
    return codes if par is None else torch.cat((codes, par.reshape(*lead[:2], -1)), -1)


def prepare(case, seed):
    layer = LAYERS[case["layer"]]
    hq, hkv, hd = layer[:3]
    act, dev = DT[case["act"]], torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    news, lens = _lengths(case)
    B, ring, sinks = case["batch"], case["ring"], case["sinks"]
    pin = (sinks + P - 1) // P * P if ring else 0
    pages = (pin + ring if ring else (max(lens) + P - 1) // P * P) // P
    n_pages = sum(pages if ring else (k + P - 1) // P for k in lens) + 5
    # pages of all sequences interleave in the pools, as in a server that runs for some time
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((B, pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(lens):
        n = pages if ring else (k + P - 1) // P
        table[b, :n] = order[at:at + n]
        at += n

    def rows():
        # about N(0, 1), with the few large elements that keys and values have
        x = torch.randn(n_pages, hkv, P, hd, generator=gen, device=dev)
        return torch.where(torch.rand(x.shape, generator=gen, device=dev) < 0.002, 8 * x, x)

    k_pool, v_pool = (_stored(layer, w, rows()).flatten() for w in (0, 1))
    th = layer[9] ** (-2 * torch.arange(hd // 2, dtype=torch.float64, device=dev) / hd)
    ang = torch.arange(max(lens) + 1, dtype=torch.float64, device=dev)[:, None] * th
    s = dict(case=dict(case), layer=layer, act=act, B=B, pages=pages, n_pages=n_pages, pin=pin, nmax=max(news), lmax=max(lens),
             news=news, table=table, k_pool=k_pool, v_pool=v_pool, rope=torch.stack((ang.cos(), ang.sin()), -1).float(),
             lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    starts = np.concatenate(([0], np.cumsum(news)))
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    if case["op"] == "read":
        # the last rows of every sequence, in order
        s["seq_ids"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(news, device=dev)).to(torch.int32)
        first = (s["lens"] - torch.tensor(news, dtype=torch.int32, device=dev))[s["seq_ids"].long()]
        s["pos"] = first + torch.arange(int(starts[-1]), dtype=torch.int32, device=dev) - s["starts"][s["seq_ids"].long()]
    else:
        # a layer whose score scale is 1 has its queries normalised: scores of a few units
        size = 1 / 8 if layer[7] else 1.0
        s["q"] = (size * torch.randn(int(starts[-1]), hq, hd, generator=gen, device=dev)).to(act)
    return s


# ---------------------------------------------------------------- the plain forms


def _gather(s, which, page, slot, to):
    """Stored rows [..., kv heads, head_dim] of pages and slots, as numbers of type `to`."""
    hkv, hd, kind, group, pt = s["layer"][1], s["layer"][2], s["layer"][3 + which], s["layer"][5], DT[s["layer"][6]]
    cb, pb = _row_bytes(s["layer"], which)
    pool = (s["v_pool"] if which else s["k_pool"]).view(s["n_pages"], hkv, P * (cb + pb))
    c = pool[..., :P * cb].unflatten(-1, (P, cb))[page, :, slot]
    if kind == "f16":
        return c.contiguous().view(torch.float16).to(to)
    par = pool[..., P * cb:].unflatten(-1, (P, pb))[page, :, slot].contiguous().view(pt).to(to)
    if kind == "sym8":
        c = c.contiguous().view(torch.int8).to(to)
    else:
        c = torch.stack((c & 15, c >> 4), -1).flatten(-2).to(to)
        if kind == "sym4":
            c = torch.where(c > 7, c - 16, c)
        elif kind == "shimmy4":
            c = c - 8
    c = c.unflatten(-1, (hd // group, group))
    if kind == "affine4":
        return (c * par[..., 0::2, None] + par[..., 1::2, None]).flatten(-2)
    return (c * par[..., None]).flatten(-2)


def _row(s, t):
    """Row of token t in its sequence's pages."""
    if not s["case"]["ring"]:
        return t
    return torch.where(t < s["pin"], t, s["pin"] + (t - s["pin"]) % s["case"]["ring"])


def _at(s, b, t):
    """(page, slot) of token t of sequence b."""
    row = _row(s, t)
    return s["table"][b, row // P].long(), row % P


def _rotated(s, x, pos):
    """RoPE of x [..., heads, head_dim] at positions pos [...]."""
    cs = s["rope"][pos].unsqueeze(-3)
    c, n = cs[..., 0], cs[..., 1]
    if s["layer"][8] == "neox":
        h = x.shape[-1] // 2
        a, b = x[..., :h], x[..., h:]
        return torch.cat((a * c - b * n, a * n + b * c), -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)


def _plain_read(s):
    page, slot = _at(s, s["seq_ids"].long(), s["pos"].long())
    return tuple(_gather(s, w, page, slot, torch.float32).to(s["act"]) for w in (0, 1))


def _plain_attention(s):
    case, layer, B, n = s["case"], s["layer"], s["B"], s["nmax"]
    hq, hkv, hd = layer[:3]
    dev, lens, starts = s["q"].device, s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    i = torch.arange(n, device=dev)
    real = i < new[:, None]                                           # [B, n]
    qpos = (lens - new)[:, None] + i
    q = s["q"][(starts[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)].float()
    q = _rotated(s, q, qpos.clamp_max(s["rope"].shape[0] - 1))
    # key positions [B, K]: all of the context, or the sinks and the tokens some window holds
    window, sinks = case["window"], case["sinks"]
    if window:
        span = torch.arange(min(window + n - 1, s["lmax"]), device=dev)
        far = lens[:, None] - span.numel() + span
        far = torch.where(far < sinks, -1, far)
        t = torch.cat((torch.arange(sinks, device=dev).expand(B, sinks), far), 1)
    else:
        t = torch.arange(s["lmax"], device=dev).expand(B, s["lmax"])
    here = (t >= 0) & (t < lens[:, None])
    page, slot = _at(s, torch.arange(B, device=dev)[:, None], torch.where(here, t, 0))
    k, v = (_gather(s, w, page, slot, torch.float32) for w in (0, 1))  # [B, K, kv heads, head_dim]
    seen = here[:, None] & real[..., None] & (t[:, None] <= qpos[..., None])
    if window:
        seen &= (t[:, None] > qpos[..., None] - window) | (t[:, None] < sinks)
    q = q.view(B, n, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, hd)
    x = q @ k.permute(0, 2, 3, 1)                                     # [B, kv heads, G * n, K]
    x = x.unflatten(2, (hq // hkv, n)) * (layer[7] or 1 / math.sqrt(hd))
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    x = x - x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    x = x.exp_()
    den = x.sum(-1, keepdim=True)
    o = x.flatten(2, 3) @ v.permute(0, 2, 1, 3)
    o = o.unflatten(2, (hq // hkv, n)) / torch.where(den == 0, 1, den)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, hq, hd).to(s["act"])
    return o[real]                                                    # the rows in order


# ---------------------------------------------------------------- the library's calls


def _handle(s):
    """What a program keeps beside its cache: the config, the output and the workspace."""
    from int8_quantized_paged_gb300 import kvq
    case, layer = s["case"], s["layer"]
    hq, hkv, hd, kk, vk, group, param, alpha, rope, base = layer
    cfg = kvq.config(hq, hkv, hd, P, kk, vk, group, group, param, param, case["act"], alpha, rope, base)
    dev, rows = s["table"].device, int(sum(s["news"]))
    h = dict(kvq=kvq, cfg=cfg, status=torch.zeros(1, dtype=torch.int32, device=dev))
    if case["op"] == "read":
        h["out"] = tuple(torch.empty(rows, hkv, hd, dtype=s["act"], device=dev) for _ in range(2))
        return h
    h["out"] = torch.empty(rows, hq, hd, dtype=s["act"], device=dev)
    if case["op"] == "sink":
        need = kvq.sink_workspace_bytes(cfg, s["B"], s["pages"], case["ring"], case["sinks"], case["window"])
    else:
        need = kvq.prefill_workspace_bytes(cfg, s["B"], rows, s["pages"], case["ring"], case["sinks"], case["window"])
    h["ws"] = torch.zeros(need, dtype=torch.uint8, device=dev)
    return h


def _own(s):
    h = s.get("handle")
    if h is None:
        h = s["handle"] = _handle(s)
    kvq, cfg, case = h["kvq"], h["cfg"], s["case"]
    if case["op"] == "read":
        kvq.read(cfg, s["seq_ids"], s["pos"], s["table"], s["B"], s["pages"], case["ring"], case["sinks"], s["k_pool"],
                 s["v_pool"], s["n_pages"], h["out"][0], h["out"][1], h["status"])
    elif case["op"] == "sink":
        kvq.sink_decode(cfg, s["q"], s["k_pool"], s["v_pool"], s["n_pages"], s["table"], s["pages"], case["ring"],
                        case["sinks"], case["window"], s["lens"], s["rope"], s["rope"].shape[0], h["out"], h["ws"],
                        h["status"])
    else:
        kvq.prefill_attention(cfg, s["q"], s["starts"], s["k_pool"], s["v_pool"], s["n_pages"], s["table"], s["pages"],
                              case["ring"], case["sinks"], case["window"], s["lens"], s["rope"], s["rope"].shape[0],
                              h["out"], h["ws"], h["status"])
    return h["out"]


def run(state):
    if own:
        return _own(state)
    return _plain_read(state) if state["case"]["op"] == "read" else _plain_attention(state)


# ---------------------------------------------------------------- what a pass cannot do without


def _seen(case, p):
    """Keys that a query at position p attends."""
    w, s = case["window"], case["sinks"]
    return p + 1 if not w or p + 1 <= w + s else w + min(s, p + 1 - w)


def work(case):
    layer = LAYERS[case["layer"]]
    hq, hkv, hd = layer[:3]
    act = 4 if case["act"] == "f32" else 2
    token = hkv * sum(sum(_row_bytes(layer, w)) for w in (0, 1))
    news, lens = _lengths(case)
    if case["op"] == "read":
        n = sum(news)
        return {"bytes": n * (token + 2 * hkv * hd * act + 8), "flops": 0}
    keys = pairs = 0
    for n, L in zip(news, lens):
        w, s = case["window"], case["sinks"]
        lo = max(0, L - n + 1 - w) if w else 0                        # the first token of the first window
        keys += L - lo + min(s, lo)
        pairs += sum(_seen(case, p) for p in range(L - n, L))
    io = sum(news) * (2 * hq * hd * act) + len(news) * 12
    return {"bytes": keys * token + io, "flops": 4 * hd * hq * pairs}


# ---------------------------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    layer, dev = s["layer"], s["table"].device
    hq, hkv, hd = layer[:3]
    news, lens = _lengths(case)
    if case["op"] == "read":
        if sum(news) * hkv * hd > 1 << 27:
            return None
        outs = []
        for which in (0, 1):
            got = []
            for b, (n, L) in enumerate(zip(news, lens)):
                t = torch.arange(L - n, L, device=dev)
                got.append(_value(s, which, b, t))
            outs.append(torch.cat(got))
        return tuple(outs)
    if sum(n * L for n, L in zip(news, lens)) * hq * hd > 1 << 39:
        return None
    at, alpha, outs = 0, layer[7] or hd ** -0.5, []
    th = torch.tensor([layer[9] ** (-2 * i / hd) for i in range(hd // 2)], dtype=torch.float64, device=dev)
    for b, (n, L) in enumerate(zip(news, lens)):
        pos = torch.arange(L - n, L, device=dev)
        q = s["q"][at:at + n].double()
        at += n
        z = torch.polar(torch.ones_like(th).expand(n, -1), pos[:, None] * th)[:, None]
        if layer[8] == "neox":
            z = z * torch.complex(q[..., :hd // 2], q[..., hd // 2:])
            q = torch.cat((z.real, z.imag), -1)
        else:
            z = z * torch.complex(q[..., 0::2], q[..., 1::2])
            q = torch.view_as_real(z).flatten(-2)
        w, first = case["window"], case["sinks"]
        t = torch.arange(L, device=dev)
        if w:
            t = t[(t < first) | (t > L - n - w)]
        k, v = _value(s, 0, b, t), _value(s, 1, b, t)
        hide = t > pos[:, None]
        if w:
            hide |= (t <= pos[:, None] - w) & (t >= first)
        out = torch.empty(n, hq, hd, dtype=torch.float64, device=dev)
        for h in range(hq):
            x = alpha * (q[:, h] @ k[:, h * hkv // hq].T)
            out[:, h] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v[:, h * hkv // hq]
        outs.append(out)
    return torch.cat(outs)


def _value(s, which, b, t):
    """Stored rows of tokens t of sequence b in 64 bits, byte by byte from the page format."""
    layer = s["layer"]
    hkv, hd, kind, group, param = layer[1], layer[2], layer[3 + which], layer[5], layer[6]
    cb, pb = _row_bytes(layer, which)
    ring, pin = s["case"]["ring"], s["pin"]
    row = t if not ring else torch.where(t < pin, t, pin + torch.remainder(t - pin, ring))
    head = torch.arange(hkv, device=t.device)
    base = (s["table"][b].long()[row // P][:, None] * hkv + head) * (P * (cb + pb))
    slot = (row % P)[:, None]
    flat = s["v_pool"] if which else s["k_pool"]
    raw = flat[(base + slot * cb)[..., None] + torch.arange(cb, device=t.device)]
    if kind == "f16":
        return raw.view(torch.float16).double()
    if kind == "sym8":
        code = raw.view(torch.int8).double()
    else:
        code = torch.empty(*raw.shape[:-1], hd, dtype=torch.float64, device=t.device)
        code[..., 0::2] = (raw % 16).double()
        code[..., 1::2] = (raw // 16).double()
        code = code - 8 if kind == "shimmy4" else torch.where(code >= 8, code - 16, code) if kind == "sym4" else code
    par = flat[(base + P * cb + slot * pb)[..., None] + torch.arange(pb, device=t.device)].view(DT[param]).double()
    if kind == "affine4":
        return code * par[..., 0::2].repeat_interleave(group, -1) + par[..., 1::2].repeat_interleave(group, -1)
    return code * par.repeat_interleave(group, -1)
