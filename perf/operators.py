"""Cases that measure the operators around the sparse-attention path: rotary
positions, the MXFP4 index cache (quantisation and indexer scores) and
eviction from the paged caches by accumulated attention weight.

Each case runs in a plain form, elementary torch operations in 32 bits (64
where 32 lose what matters), or, with ``own`` true, through the framework's
entry points.  ``exact`` gives the computed outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 64
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MASS_BITS = 40
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # One decode step's attention queries: the rope part of each head, a slice of the up-projection's
        # output, is rotated into the last 64 of the 576 query dims.  Positions deep in a 128K context.
        _rope("rope_decode_query", T=8, H=128, D=64, src=192, dst=576, rot=64, offset=0, interleaved=True,
              scaling="yarn", factor=32.0, dtype="bf16", transpose=False, top=131072, run=False),
        # The index queries of one long prefill chunk: 64 rotated dims of 128 in the half layout, the others copied.
        _rope("rope_prefill_index_query", T=8192, H=64, D=128, src=128, dst=128, rot=64, offset=64, interleaved=False,
              scaling="linear", factor=4.0, dtype="bf16", transpose=False, top=65536, run=True),
        # The gradient of a training step's rotated queries, in fp32 and with an odd token count.
        _rope("rope_gradient_fp32", T=2047, H=16, D=64, src=64, dst=64, rot=64, offset=0, interleaved=True,
              scaling="none", factor=1.0, dtype="fp32", transpose=True, top=2047, run=True),
        # One decode step: 8 index queries and the 8 new keys into the cache.
        dict(name="mx4_quantize_decode", op="quantize", B=8, q=1, ctx=255, step=3),
        # A chunk of 16 prompts: 4096 index queries, and their keys written through the page table.
        dict(name="mx4_quantize_chunk", op="quantize", B=16, q=256, ctx=1500, step=37),
        # A short decode batch, where launches and latency count.
        dict(name="mx4_scores_decode_short", op="scores", B=3, q=1, ctx=1000, step=171),
        # The long decode step: 8 sequences of 128K cached keys.
        dict(name="mx4_scores_decode_8x128k", op="scores", B=8, q=1, ctx=131072, step=0),
        # Two prompt chunks of 1000 queries against ragged contexts of about 8K.
        dict(name="mx4_scores_prefill", op="scores", B=2, q=1000, ctx=8191, step=1030),
        # A decode step's attention weights: 8 sequences, 2048 selected rows each, 128 heads.
        dict(name="mass_decode_8x128k", op="mass", B=8, q=1, ctx=131072, step=0, K=2048, H=128, kv="bf16"),
        # A prompt chunk over the FP8 latent cache, 64 heads; early tokens have fewer candidates than slots.
        dict(name="mass_prefill_fp8", op="mass", B=2, q=200, ctx=2300, step=331, K=2048, H=64, kv="fp8"),
        # One short sequence over its budget.
        dict(name="evict_one", op="evict", B=1, ctx=3001, step=0, budget=1024, recent=64, sink=4, kv="fp8"),
        # A batch of 8 long contexts cut back to a quarter.
        dict(name="evict_8x32k", op="evict", B=8, ctx=32768, step=517, budget=8192, recent=256, sink=4, kv="bf16"),
    ]


def _rope(name, **kw):
    return dict(name=name, op="rope", theta=10000.0, original=4096, **kw)


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "quantize", "scores", "scores", "mass", "evict"])
    if op == "rope":
        rot = rng.choice([32, 64, 64, 128])
        rest = rng.choice([0, 0, 32, 64])
        D = rot + rest
        T = _log(rng, 1, 8192)
        H = rng.choice([1, 3, 16, 64, 128])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        while T * H * D * (4 if dtype == "fp32" else 2) > 8192 * 64 * 256:
            T = max(1, T // 2 - 1)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op="rope", theta=rng.choice([10000.0, 500000.0]), original=4096, T=T, H=H, D=D,
                    src=D + rng.choice([0, 0, 128]), dst=D + rng.choice([0, 0, 512]), rot=rot,
                    offset=rng.choice([0, rest]), interleaved=rng.random() < 0.5, scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                    dtype=dtype, transpose=rng.random() < 0.4,
                    top=T + _log(rng, 1, 131072), run=rng.random() < 0.7)
    if op == "quantize":
        B = rng.randint(1, 16)
        q = _log(rng, 1, 256)
        return dict(op="quantize", B=B, q=q, ctx=q + _log(rng, 1, 1200), step=rng.randint(0, 63))
    if op == "scores":
        if rng.random() < 0.5:                       # decode
            B = rng.randint(1, 8)
            ctx = _log(rng, 1, 131072)
            return dict(op="scores", B=B, q=1, ctx=ctx, step=rng.randint(0, max(1, ctx // B)))
        B = rng.randint(1, 3)
        q = _log(rng, 2, 600)
        return dict(op="scores", B=B, q=q, ctx=q + _log(rng, 1, 7000), step=rng.randint(0, 200))
    if op == "mass":
        H = rng.choice([16, 32, 64, 128])
        kv = rng.choice(["bf16", "fp8"])
        K = _log(rng, 17, 2048)
        if rng.random() < 0.5:
            B = rng.randint(1, 8)
            ctx = _log(rng, 1, 100000)
            return dict(op="mass", B=B, q=1, ctx=ctx, step=rng.randint(0, max(1, ctx // B)), K=K, H=H, kv=kv)
        B = rng.randint(1, 3)
        q = _log(rng, 2, 60)
        return dict(op="mass", B=B, q=q, ctx=q + _log(rng, 1, 6000), step=rng.randint(0, 60), K=K, H=H, kv=kv)
    B = rng.randint(1, 8)
    ctx = _log(rng, 300, 32768)
    budget = _log(rng, 64, max(65, ctx // 4))
    return dict(op="evict", B=B, ctx=ctx, step=rng.randint(0, ctx // (2 * B)), budget=budget,
                recent=rng.randint(0, budget // 4), sink=rng.randint(0, 8), kv=rng.choice(["bf16", "fp8"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _lengths(c):
    """ctx_len of each sequence: ragged by `step`, never below its query tokens."""
    return [max(c.get("q", 1), c["ctx"] - b * c["step"]) for b in range(c["B"])]


def _geometry(c, g, spare_pages=0):
    ctx = _lengths(c)
    B, q = c["B"], c.get("q", 1)
    pages = [(n + PAGE - 1) // PAGE for n in ctx]
    total = sum(pages) + spare_pages
    perm = torch.randperm(total, generator=g, device=DEV)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n].int()
        at += n
    s = {"ctx": torch.tensor(ctx, dtype=torch.int32, device=DEV), "table": table, "num_pages": total,
         "starts": torch.arange(0, B * q + 1, q, dtype=torch.int32, device=DEV), "max_ctx": max(ctx), "T": B * q,
         "spare": perm[at:].int()}
    s["pos"] = (s["ctx"].long()[:, None] - q + torch.arange(q, device=DEV)).reshape(-1)       # [T]
    s["seq"] = torch.arange(B, device=DEV).repeat_interleave(q)
    if own:
        import sparse_indexed_attention_b200 as dsa
        s["seqs"] = dsa.Seqs(s["starts"], s["ctx"], table, total, s["max_ctx"], B * q)
    return s


def _rows(table, b, s):
    """Pool rows of logical positions s of sequences b."""
    return table[b, s // PAGE].long() * PAGE + s % PAGE


def _inv_freq(c):
    """Rotation per position of each pair, in radians (64 bits)."""
    rot, theta, f = c["rot"], c["theta"], c["factor"]
    j = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    if c["scaling"] == "ntk":
        theta = theta * f ** (rot / (rot - 2))
    base = theta ** (-2.0 * j / rot)
    if c["scaling"] == "linear":
        base = base / f
    if c["scaling"] == "yarn":
        dim = lambda turns: rot * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = ((j - low) / max(high - low, 0.001)).clamp(0, 1)
        base = base / f * ramp + base * (1 - ramp)
    return base


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0


def _quantize(x):
    """MXFP4 of [..., 128] values: E2M1 codes [..., 128] (sign in bit 3) and exponents [..., 4]."""
    b = x.float().unflatten(-1, (4, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, (torch.frexp(amax).exponent - 3).clamp(-127, 127), 0)
    y = torch.ldexp(b.abs(), -e[..., None])
    code = ((y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    return (code + 8 * (b < 0)).flatten(-2).byte(), e


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(codes, e):
    """What codes and exponents stand for, fp32."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    return torch.ldexp(t[codes.int()].unflatten(-1, (4, 32)), e[..., None]).flatten(-2)


def _unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def _fp8_latent(x):
    """E4M3 codes [R, 576] and tile-scale bytes [R, 8]: one power of two per 128 values."""
    t = torch.nn.functional.pad(x, (0, 64)).unflatten(-1, (5, 128))
    a = t.abs().amax(-1)
    e = torch.where(a > 0, torch.ceil(torch.log2(a / 448.0)), 0).int()
    codes = torch.ldexp(t, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.zeros((x.shape[0], 8), dtype=torch.uint8, device=x.device)
    scale[:, :5] = (e + 127).byte()
    return codes.flatten(-2)[:, :576].contiguous(), scale


def _latent(kv, kv_scale, rows):
    """fp32 latent rows of the pool."""
    if kv_scale is None:
        return kv[rows].float()
    v = kv[rows].view(torch.float8_e4m3fn).float()
    e = (kv_scale[rows][..., :5].int() - 127).repeat_interleave(128, -1)[..., :576]
    return torch.ldexp(v, e)


def prepare(case, seed):
    c = case
    g = torch.Generator(DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if c["op"] == "rope":
        T, H, D, dt = c["T"], c["H"], c["D"], DTYPES[c["dtype"]]
        x = randn(T, H, c["src"]).to(dt)[..., c["src"] - D:]
        out = torch.zeros((T, H, c["dst"]), dtype=dt, device=DEV)[..., c["dst"] - D:]
        if c["run"]:
            pos = torch.arange(c["top"] - T, c["top"], device=DEV)
        else:
            pos = torch.randint(c["top"] // 2, c["top"], (T,), generator=g, device=DEV)
        s = {"x": x, "out": out, "pos": pos, "inv_freq": _inv_freq(c), "amp": _amplitude(c)}
        if own:
            import sparse_indexed_attention_b200 as dsa
            s["table"] = dsa.RopeTable.build(c["rot"], c["theta"], interleaved=c["interleaved"], scaling=c["scaling"],
                                             factor=c["factor"], original_max=c["original"], device=DEV)
    elif c["op"] == "quantize":
        s = _geometry(c, g)
        s["qI"] = randn(s["T"], 64, 128).bfloat16()
        s["k"] = randn(s["T"], 128).bfloat16()
        s["kI"] = torch.zeros((s["num_pages"] * PAGE, 64), dtype=torch.uint8, device=DEV)
        s["kI_scale"] = torch.full((s["num_pages"] * PAGE, 4), 127, dtype=torch.uint8, device=DEV)
    elif c["op"] == "scores":
        s = _geometry(c, g)
        R = s["num_pages"] * PAGE
        codes, e = _quantize(randn(R, 128))
        s["kI"], s["kI_scale"] = _pack(codes), (e + 127).byte()
        s["qI"] = randn(s["T"], 64, 128).bfloat16()
        s["w"] = randn(s["T"], 64) / 8
        s["scores"] = torch.zeros((s["T"], (s["max_ctx"] + 3) // 4 * 4), device=DEV)
    elif c["op"] == "mass":
        s = _geometry(c, g)
        R, T, K = s["num_pages"] * PAGE, s["T"], c["K"]
        kv = randn(R, 576)
        kv *= torch.where(torch.rand((R, 1), generator=g, device=DEV) < 0.01, 3.0, 1.0)   # a few rows that stand out
        s["kv"], s["kv_scale"] = (kv.bfloat16(), None) if c["kv"] == "bf16" else _fp8_latent(kv)
        del kv
        s["q"] = randn(T, c["H"], 576).bfloat16()
        # K distinct causal positions of each token, ascending, -1 behind them
        n = s["max_ctx"]
        key = torch.rand((T, n), generator=g, device=DEV)
        key = torch.where(torch.arange(n, device=DEV) <= s["pos"][:, None], key, 2.0)
        order = key.argsort(dim=1)[:, :min(K, n)]
        order = torch.where(order <= s["pos"][:, None], order, n).sort(dim=1).values
        s["idx"] = torch.full((T, K), -1, dtype=torch.int32, device=DEV)
        s["idx"][:, :order.shape[1]] = torch.where(order < n, order, -1).int()
        s["scale"] = 576 ** -0.5
        s["lse"] = torch.logsumexp(_logits(s, torch.float64), dim=-1).float()
        s["mass"] = torch.zeros((c["B"], n), dtype=torch.int64, device=DEV)
    else:
        new = (min(c["budget"], max(_lengths(c))) + PAGE - 1) // PAGE
        s = _geometry(c, g, spare_pages=c["B"] * new)
        R = s["num_pages"] * PAGE
        s["new_table"] = s["spare"].reshape(c["B"], new).contiguous()
        x = randn(R, 576)
        s["pools"] = [x.bfloat16()] if c["kv"] == "bf16" else list(_fp8_latent(x))
        del x
        s["pools"] += [torch.randint(0, 256, (R, n), generator=g, device=DEV, dtype=torch.uint8) for n in (64, 4)]
        # heavy-tailed weights, a third of the positions never attended to
        m = torch.exp(3.0 * randn(c["B"], s["max_ctx"])) * 2.0 ** (MASS_BITS - 12)
        s["mass"] = torch.where(torch.rand(m.shape, generator=g, device=DEV) < 0.33, 0.0, m).long()
        s["new_mass"] = torch.zeros((c["B"], new * PAGE), dtype=torch.int64, device=DEV)
    s["case"] = c
    return s


# ---------------------------------------------------------------------------
# the pass
# ---------------------------------------------------------------------------


def _logits(s, dtype):
    """scale * q . KV over the selected rows, [T, H, K]; -inf where a slot is unused."""
    idx = s["idx"].long()
    rows = _rows(s["table"], s["seq"][:, None], idx.clamp(min=0))
    kv = _latent(s["kv"], s["kv_scale"], rows).to(dtype)
    logits = torch.einsum("thd,tkd->thk", s["q"].to(dtype), kv) * s["scale"]
    return logits.masked_fill(idx[:, None, :] < 0, -math.inf)


def run(state):
    s, c = state, state["case"]
    return (_own if own else _plain)(s, c)


def _own(s, c):
    import sparse_indexed_attention_b200 as dsa
    if c["op"] == "rope":
        return dsa.dsa_rope(s["x"], s["pos"], s["table"], offset=c["offset"], out=s["out"], transpose=c["transpose"])
    if c["op"] == "quantize":
        codes, scales = dsa.dsa_quantize_index_query_mx4(s["qI"])
        dsa.dsa_append_index_keys_mx4(s["seqs"], s["k"], s["kI"], s["kI_scale"])
        return dsa.dsa_dequantize_mx4(codes, scales), dsa.dsa_dequantize_mx4(s["kI"], s["kI_scale"])
    if c["op"] == "scores":
        return dsa.dsa_index_scores(s["seqs"], s["qI"], s["w"], s["kI"], s["kI_scale"], scores=s["scores"])
    if c["op"] == "mass":
        s["mass"].zero_()                            # a request's first step
        dsa.dsa_attn_mass(s["seqs"], s["q"], s["kv"], s["idx"], s["lse"], s["scale"], s["mass"],
                          kv_scale=s["kv_scale"])
        return s["mass"] * 2.0 ** -MASS_BITS
    keep, keep_len = dsa.dsa_evict_select(s["ctx"], s["mass"], c["budget"], recent=c["recent"], sink=c["sink"])
    dsa.dsa_evict_compact(s["seqs"], keep, keep_len, s["new_table"], s["pools"], mass=s["mass"],
                          new_mass=s["new_mass"])
    return [keep, keep_len, s["new_mass"], *s["pools"]]


def _plain(s, c):
    if c["op"] == "rope":
        return _plain_rope(s, c)
    if c["op"] == "quantize":
        qI = _values(*_quantize(s["qI"])).bfloat16()
        codes, e = _quantize(s["k"])
        rows = _rows(s["table"], s["seq"], s["pos"])
        s["kI"][rows] = _pack(codes)
        s["kI_scale"][rows] = (e + 127).byte()
        return qI, _values(_unpack(s["kI"]), s["kI_scale"].int() - 127).bfloat16()
    if c["op"] == "scores":
        return _plain_scores(s, c)
    if c["op"] == "mass":
        logits = _logits(s, torch.float32)
        weight = torch.exp(logits - s["lse"][..., None]).mean(1)
        mass = torch.zeros(s["mass"].numel(), dtype=torch.float64, device=DEV)
        at = s["seq"][:, None] * s["mass"].shape[1] + s["idx"].long().clamp(min=0)
        mass.index_add_(0, at.flatten(), weight.double().flatten())
        return mass.float().view(s["mass"].shape)
    return _plain_evict(s, c)


def _plain_rope(s, c):
    rot, o = c["rot"], c["offset"]
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = ((f(angle) * s["amp"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    sin = -sin if c["transpose"] else sin
    x = s["x"].float()
    r = x[..., o:o + rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :rot // 2], r[..., rot // 2:])
    y = [a * cos - b * sin, a * sin + b * cos]
    y = torch.stack(y, -1).flatten(-2) if c["interleaved"] else torch.cat(y, -1)
    s["out"].copy_(torch.cat([x[..., :o], y, x[..., o + rot:]], -1))
    return s["out"]


def _plain_scores(s, c):
    B, q, n = c["B"], c["q"], s["max_ctx"]
    at = torch.arange(n, device=DEV)
    live = at < s["ctx"][:, None]
    rows = _rows(s["table"], torch.arange(B, device=DEV)[:, None], torch.where(live, at, 0))
    keys = _values(_unpack(s["kI"][rows]), s["kI_scale"][rows].int() - 127)              # [B, n, 128]
    qI = _values(*_quantize(s["qI"])).view(B, q * 64, 128)
    dots = torch.matmul(qI, keys.transpose(1, 2)).view(B, q, 64, n).clamp_(min=0)
    score = torch.matmul(s["w"].view(B, q, 1, 64), dots).view(B * q, n)
    s["scores"][:, :n] = torch.where(at <= s["pos"][:, None], score, 0.0)
    return s["scores"]


def _plain_evict(s, c):
    n, budget = s["max_ctx"], c["budget"]
    at, ctx = torch.arange(n, device=DEV), s["ctx"].long()[:, None]
    key = s["mass"].float()                          # weights are compared in 24 bits, ties to the lower position
    key = torch.where((at < c["sink"]) | (at >= ctx - c["recent"]), math.inf, key)
    key = torch.where(at < ctx, key, -math.inf)
    order = key.sort(dim=1, descending=True, stable=True).indices[:, :min(budget, n)]
    order = torch.where(order < ctx, order, n).sort(dim=1).values
    keep = torch.full((c["B"], budget), -1, dtype=torch.int32, device=DEV)
    keep[:, :order.shape[1]] = torch.where(order < n, order, -1).int()
    keep_len = ctx[:, 0].clamp(max=budget).int()
    b, i = (keep >= 0).nonzero(as_tuple=True)
    old = keep[b, i].long()
    src, dst = _rows(s["table"], b, old), _rows(s["new_table"], b, i)
    for pool in s["pools"]:
        pool[dst] = pool[src]
    s["new_mass"][b, i] = s["mass"][b, old]
    return [keep, keep_len, s["new_mass"], *s["pools"]]


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the outputs in 64 bits
# ---------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["H"]
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * c["D"] * size + 8 * c["T"] + 4 * c["rot"], "flops": 3 * n * c["rot"]}
    ctx = _lengths(c)
    q = c.get("q", 1)
    T = c["B"] * q
    if c["op"] == "quantize":
        pool = sum((n + PAGE - 1) // PAGE for n in ctx) * PAGE
        return {"bytes": T * 65 * (256 + 68) + T * 64 * (68 + 256) + pool * (68 + 256), "flops": 2 * T * 65 * 128}
    if c["op"] == "scores":
        pairs = sum(q * n - q * (q - 1) // 2 for n in ctx)
        return {"bytes": 68 * sum(ctx) + T * 64 * (256 + 4) + 4 * pairs, "flops": pairs * 64 * (2 * 128 + 3)}
    if c["op"] == "mass":
        row = 1152 if c["kv"] == "bf16" else 584
        picked = [[min(c["K"], n - q + j + 1) for j in range(q)] for n in ctx]
        rows = sum(min(n, sum(p)) for n, p in zip(ctx, picked))
        pairs = sum(map(sum, picked)) * c["H"]
        return {"bytes": rows * row + T * c["H"] * (1152 + 4) + 4 * T * c["K"] + 8 * rows, "flops": pairs * (2 * 576 + 3)}
    kept = sum(min(c["budget"], n) for n in ctx)
    row = (1152 if c["kv"] == "bf16" else 584) + 64 + 4 + 8
    return {"bytes": 8 * sum(ctx) + 4 * c["B"] * c["budget"] + 2 * kept * row, "flops": sum(ctx)}


def _grid4(x):
    """MXFP4 values of x [..., 128] by a search of the grid, in 64 bits: nearest, ties to the even code."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for k in range(4):
        v = x[..., 32 * k:32 * k + 32].double()
        top = v.abs().max(-1, keepdim=True).values
        unit = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2)
        y = (v.abs() / unit).clamp(max=6.0)
        best, far = torch.zeros_like(y), y.clone()
        for i in range(1, 8):
            d = (y - grid[i]).abs()
            take = (d < far) | ((d == far) & (i % 2 == 0))
            best, far = torch.where(take, grid[i], best), torch.where(take, d, far)
        out[..., 32 * k:32 * k + 32] = torch.copysign(best, v) * unit
    return out


def exact(case, seed):
    c = case
    if c["op"] == "evict":
        return None                                  # moves and comparisons, nothing computed
    s = prepare(c, seed)
    if c["op"] == "rope":
        z = s["x"].double().clone()
        half = c["rot"] // 2
        turn = torch.polar(torch.full((c["T"], half), float(s["amp"]), dtype=torch.float64, device=DEV),
                           torch.outer(s["pos"].double(), s["inv_freq"]))
        turn = turn.conj() if c["transpose"] else turn
        for j in range(half):
            i0, i1 = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
            v = torch.complex(z[..., c["offset"] + i0], z[..., c["offset"] + i1]) * turn[:, j:j + 1]
            z[..., c["offset"] + i0], z[..., c["offset"] + i1] = v.real, v.imag
        return z
    table, ctx, q = s["table"].long(), _lengths(c), c["q"]
    if c["op"] == "quantize":
        pool = torch.zeros((s["num_pages"] * PAGE, 128), dtype=torch.float64, device=DEV)
        k = _grid4(s["k"])
        for b, n in enumerate(ctx):
            at = torch.arange(n - q, n, device=DEV)
            pool[table[b][at // PAGE] * PAGE + at % PAGE] = k[b * q:(b + 1) * q]
        return _grid4(s["qI"]), pool
    if c["op"] == "scores":
        value = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)
        qI, out = _grid4(s["qI"]), torch.zeros(s["scores"].shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(ctx):
            at = torch.arange(n, device=DEV)
            row = table[b][at // PAGE] * PAGE + at % PAGE
            raw = s["kI"][row].long()
            key = torch.empty((n, 128), dtype=torch.float64, device=DEV)
            key[:, 0::2], key[:, 1::2] = value[raw % 16], value[raw // 16]
            key *= torch.exp2(s["kI_scale"][row].double() - 127).repeat_interleave(32, 1)
            for t0 in range(b * q, (b + 1) * q, 64):
                t1 = min(t0 + 64, (b + 1) * q)
                dots = torch.relu(qI[t0:t1].reshape(-1, 128) @ key.T).view(t1 - t0, 64, n)
                out[t0:t1, :n] = (s["w"][t0:t1].double()[..., None] * dots).sum(1) * (at <= s["pos"][t0:t1, None])
        return out
    mass = torch.zeros(s["mass"].shape, dtype=torch.float64, device=DEV)
    for t in range(s["T"]):
        b = t // q
        at = s["idx"][t][s["idx"][t] >= 0].long()
        row = table[b][at // PAGE] * PAGE + at % PAGE
        if s["kv_scale"] is None:
            kv = s["kv"][row].double()
        else:
            kv = s["kv"][row].view(torch.float8_e4m3fn).to(torch.float32).double()
            kv = kv * torch.exp2(s["kv_scale"][row].double() - 127).repeat_interleave(128, 1)[:, :576]
        p = torch.exp(s["scale"] * (s["q"][t].double() @ kv.T) - s["lse"][t].double()[:, None])
        mass[b, at] += p.sum(0) / c["H"]
    return mass
