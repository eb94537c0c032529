"""The operators between the quantized linears of a diffusion-transformer block,
as cases to measure: the norm fused with the gate and residual before it, rotary
positions with the query/key norm, attention over an encoder's states, and the
low-rank adapters of many requests beside a shared projection.

`run` is one call of an operator.  With `own` false it is the plain form:
elementary torch operations in 32 bits (angles in 64), rounded once at the end.
With `own` true it is the call a user makes of nvfp4_block_scaled_05_amd.
`exact` is the definition in 64 bits, written apart from both.

Sizes: hidden 3072, 24 heads of 128, MLP 12288, 16384 or 4096 image tokens and 512
text tokens are the repository's own DiT workloads; the rest are generic.
"""

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def listed():
    return [
        # The second norm of a block at 2048^2: attention output gated into the residual stream,
        # LayerNorm, scale and shift from the modulation linear's [batch, 6 * hidden] output, the
        # amax for the quantizer that follows.
        {"name": "norm-block-2048", "op": "norm", "batch": 1, "tokens": 16896, "channels": 3072,
         "stream": "bf16", "norm": "layer", "post": "none", "modulated": True, "weights": False,
         "residual_scale": 1.0, "amax": True},
        # Norms before and after a block around an fp32 residual stream: three ragged prompts,
        # RMS norms with weights, the residual scaled.
        {"name": "norm-sandwich-f32", "op": "norm", "batch": 3, "tokens": 1021, "channels": 1536,
         "stream": "f32", "norm": "rms", "post": "rms", "modulated": True, "weights": True,
         "residual_scale": 0.75, "amax": False},
        # One pooled token a request: a call whose launch is its cost.
        {"name": "norm-tokens", "op": "norm", "batch": 4, "tokens": 1, "channels": 3072,
         "stream": "bf16", "norm": "layer", "post": "none", "modulated": True, "weights": False,
         "residual_scale": 1.0, "amax": False},
        # Queries and keys of the block at 2048^2, views of the fused QKV projection, with the
        # query/key norm and three position axes (text index, image row, image column).
        {"name": "rotary-qkv-2048", "op": "rotary", "batch": 1, "tokens": 16896, "heads": 24,
         "kv_heads": 24, "dim": 128, "rotary_dim": 128, "axes": "16 56 56", "layout": "interleaved",
         "scaling": "none", "factor": 1.0, "original": 0, "far": 128, "norm": True},
        # A text encoder far past its trained length: half layout, half of each head, shared key
        # heads, positions to 131071 with the by-parts scaling.
        {"name": "rotary-long-yarn", "op": "rotary", "batch": 2, "tokens": 2039, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary_dim": 64, "axes": "", "layout": "half",
         "scaling": "yarn", "factor": 32.0, "original": 4096, "far": 131071, "norm": False},
        # One new token for each of 16 requests.
        {"name": "rotary-tokens", "op": "rotary", "batch": 16, "tokens": 1, "heads": 24,
         "kv_heads": 24, "dim": 64, "rotary_dim": 64, "axes": "", "layout": "half",
         "scaling": "linear", "factor": 4.0, "original": 0, "far": 8191, "norm": False},
        # Image queries of a CFG pair at 2048^2 over the encoder's 512 text states; the
        # unconditional prompt is short.
        {"name": "attn-text-2048", "op": "attn", "batch": 2, "queries": 16384, "keys": 512,
         "heads": 24, "kv_heads": 24, "dim": 128, "lengths": "512 77", "keep": 1.0},
        # Image queries at 1024^2 over image and text states together.
        {"name": "attn-joint-1024", "op": "attn", "batch": 1, "queries": 4096, "keys": 4608,
         "heads": 24, "kv_heads": 24, "dim": 128, "lengths": "", "keep": 1.0},
        # Three requests with holes in their key masks (one has no key left), shared key heads,
        # 64-wide heads, odd lengths, undefined values under the mask.
        {"name": "attn-mask-shared", "op": "attn", "batch": 3, "queries": 1021, "keys": 1301,
         "heads": 16, "kv_heads": 4, "dim": 64, "lengths": "1301 900 0", "keep": 0.8},
        # One query token for each of 8 requests over long states of their own.
        {"name": "attn-token-long", "op": "attn", "batch": 8, "queries": 1, "keys": 8192,
         "heads": 24, "kv_heads": 8, "dim": 128, "lengths": "8192 8191 6000 4097 4096 1000 33 1",
         "keep": 1.0},
        # Adapters of four requests beside the QKV projection at 1024^2.
        {"name": "lora-qkv-1024", "op": "lora", "rows": 4608, "inner": 3072, "outer": 9216,
         "rank": 32, "adapters": 4, "requests": 5, "epilogue": "none", "amax": False},
        # 48 rows of 12 requests through the up projection, the GELU and its amax after the adapters.
        {"name": "lora-up-few", "op": "lora", "rows": 48, "inner": 3072, "outer": 12288,
         "rank": 16, "adapters": 8, "requests": 12, "epilogue": "gelu", "amax": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rotary", "attn", "lora"])
    if op == "norm":
        channels = 8 * _log(rng, 8, 1024)
        batch = rng.randint(1, 4)
        tokens = _log(rng, 1, min(8192, 50_000_000 // (batch * channels)))
        return {"op": op, "batch": batch, "tokens": tokens, "channels": channels,
                "stream": rng.choice(["bf16", "f32"]), "norm": rng.choice(["layer", "rms"]),
                "post": rng.choice(["none", "none", "rms", "layer"]),
                "modulated": rng.random() < 0.75, "weights": rng.random() < 0.5,
                "residual_scale": rng.choice([1.0, 0.5]), "amax": rng.random() < 0.5}
    if op == "rotary":
        dim = 16 * rng.randint(2, 8)
        kv_heads = rng.randint(1, 8)
        heads = kv_heads * rng.randint(1, 4)
        batch = rng.randint(1, 8)
        tokens = _log(rng, 1, min(16384, 100_000_000 // (batch * (heads + kv_heads) * dim)))
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "rotary_dim": 16 * rng.randint(1, dim // 16), "axes": "",
                "layout": rng.choice(["interleaved", "half"]), "scaling": scaling,
                "factor": 1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                "original": 4096 if scaling == "yarn" else 0, "far": _log(rng, 16, 131071),
                "norm": rng.random() < 0.5}
    if op == "attn":
        dim = rng.choice([64, 64, 80, 96, 128, 128])
        kv_heads = rng.randint(1, 8)
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        batch = rng.randint(1, 4)
        queries = 1 if rng.random() < 0.3 else _log(rng, 2, 4096)
        most = 20_000_000_000 // (batch * heads * queries * dim)
        keys = _log(rng, 1, max(1, min(16384, most)))
        lengths = "" if rng.random() < 0.4 else " ".join(
            str(rng.choice([keys, rng.randint(0, keys)])) for _ in range(batch))
        return {"op": op, "batch": batch, "queries": queries, "keys": keys, "heads": heads,
                "kv_heads": kv_heads, "dim": dim, "lengths": lengths,
                "keep": rng.choice([1.0, 1.0, 0.9, 0.5])}
    inner, outer = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 1536)
    return {"op": op, "rows": _log(rng, 1, 4096), "inner": inner, "outer": outer,
            "rank": 8 * rng.randint(1, 8), "adapters": rng.randint(1, 8),
            "requests": rng.randint(1, 16), "epilogue": rng.choice(["none", "none", "gelu"]),
            "amax": rng.random() < 0.3}


def _numbers(text):
    return [int(v) for v in text.split()]


def _lengths(case):
    return _numbers(case["lengths"]) or [case["keys"]] * case["batch"]


def _frequencies(case):
    """Angle per position of each rotary pair (radians, 64 bits), the position axis of each
    pair, and the factor on the rotated values.  Linear: angles divided by the factor.  NTK:
    the base raised so the slowest pair's angle is divided by it.  YaRN by parts: pairs that
    turn less than once over the trained length are divided, those that turn more than 32
    times are kept, those between are blended linearly in the pair index; values are scaled
    by 0.1 ln(factor) + 1."""
    base, factor, rot = 10000.0, case["factor"], case["rotary_dim"]
    dims = _numbers(case["axes"]) or [rot]
    freq, axis = [], []
    for a, d in enumerate(dims):
        b = base
        if case["scaling"] == "ntk" and d > 2:
            b = base * factor ** (d / (d - 2))
        for j in range(d // 2):
            f = b ** (-2.0 * j / d)
            if case["scaling"] == "linear":
                f /= factor
            if case["scaling"] == "yarn":
                def pair_at(turns):
                    return d * math.log(case["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
                low = max(math.floor(pair_at(32.0)), 0)
                high = min(math.ceil(pair_at(1.0)), d - 1)
                if high == low:
                    high += 0.001
                slow = min(max((j - low) / (high - low), 0.0), 1.0)
                f = f * (1 - slow) + f / factor * slow
            freq.append(f)
            axis.append(a)
    magnitude = 0.1 * math.log(factor) + 1.0 if case["scaling"] == "yarn" and factor > 1 else 1.0
    return freq, axis, magnitude


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=BF16):
        return (torch.randn(shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    s = {"case": case}
    if case["op"] == "norm":
        b, t, c = case["batch"], case["tokens"], case["channels"]
        stream = BF16 if case["stream"] == "bf16" else F32
        # a residual stream whose channels have means and sizes of their own
        s["x"] = (normal(b, t, c, dtype=F32) * normal(c, std=2.0, dtype=F32) + normal(c, dtype=F32)).to(stream)
        s["y"] = normal(b, t, c)
        # shift, scale and gate as the modulation linear lays them out, side by side
        mod = normal(b, 6 * c, std=0.3)
        s["shift"], s["scale"], s["gate"] = (
            (mod[:, :c], mod[:, c:2 * c], mod[:, 2 * c:3 * c]) if case["modulated"] else (None,) * 3)
        s["weight"] = 1 + normal(c, std=0.1, dtype=F32) if case["weights"] else None
        s["bias"] = normal(c, std=0.1, dtype=F32) if case["weights"] and case["norm"] == "layer" else None
        s["post_weight"] = 1 + normal(c, std=0.1, dtype=F32) if case["weights"] and case["post"] != "none" else None
        s["amax"] = torch.empty(1, dtype=F32, device="cuda") if case["amax"] else None
    elif case["op"] == "rotary":
        b, t, h, hk, d = (case[n] for n in ("batch", "tokens", "heads", "kv_heads", "dim"))
        # the fused projection's output: query heads, key heads, value heads of each token
        qkv = normal(b, t, h + 2 * hk, d)
        s["q"], s["k"] = qkv[:, :, :h], qkv[:, :, h:h + hk]
        axes = len(_numbers(case["axes"])) or 1
        s["positions"] = whole(0, case["far"] + 1, b, t, axes) if axes > 1 else whole(0, case["far"] + 1, b, t)
        s["q_weight"] = 1 + normal(d, std=0.1, dtype=F32) if case["norm"] else None
        s["k_weight"] = 1 + normal(d, std=0.1, dtype=F32) if case["norm"] else None
        freq, axis, s["magnitude"] = _frequencies(case)
        s["freq"] = torch.tensor(freq, dtype=F64, device="cuda")
        s["axis"] = torch.tensor(axis, dtype=torch.int64, device="cuda")
        if own:
            import nvfp4_block_scaled_05_amd as nv
            s["plan"] = nv.rotary_plan(case["rotary_dim"], axes=_numbers(case["axes"]) or None,
                                       scaling=case["scaling"], factor=case["factor"],
                                       original_length=case["original"])
    elif case["op"] == "attn":
        b, lq, lk, h, hk, d = (case[n] for n in ("batch", "queries", "keys", "heads", "kv_heads", "dim"))
        s["q"] = normal(b, lq, h, d)
        # keys and values side by side, as the encoder's projection writes them
        kv = normal(b, lk, 2, hk, d)
        lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        at = torch.arange(lk, device="cuda")
        visible = at[None, :] < lengths[:, None]
        s["lengths"] = lengths if case["lengths"] else None
        s["mask"] = None
        if case["keep"] < 1:
            s["mask"] = torch.rand((b, lk), generator=g, device="cuda").argsort(1) < int(case["keep"] * lk)
            visible = visible & s["mask"]
        # what lies in masked places is undefined
        kv[~visible] = float("nan")
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    else:
        t, k, n, r, m = (case[c] for c in ("rows", "inner", "outer", "rank", "adapters"))
        s["x"], s["y"] = normal(t, k), normal(t, n)
        s["down"] = normal(m, r, k, std=k ** -0.5)
        s["up"] = normal(m, n, r, std=0.5 * r ** -0.5)
        s["scales"] = 0.5 + torch.rand(m, generator=g, device="cuda", dtype=F32)
        # rows of one request lie together; one request in eight has no adapter
        cuts = whole(0, t + 1, case["requests"] - 1).sort().values
        request = torch.bucketize(torch.arange(t, device="cuda", dtype=torch.int32), cuts, right=True)
        of = whole(0, m, case["requests"])
        of[whole(0, 8, case["requests"]) == 0] = -1
        s["ids"] = of[request].contiguous()
        s["amax"] = torch.empty(1, dtype=F32, device="cuda") if case["amax"] else None
    return s


# ------------------------------------------------------------------ the calls

def _bf16_of(amax):
    """The amax of bf16 values as the bf16 number it is: the upper half of its fp32 word."""
    return None if amax is None else amax.view(BF16)[1:]


def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_norm(s):
    import nvfp4_block_scaled_05_amd as nv
    c = s["case"]
    r, h = nv.gated_norm(s["x"], s["y"], gate=s["gate"], scale=s["scale"], shift=s["shift"],
                         norm=c["norm"], weight=s["weight"], bias=s["bias"], post_norm=c["post"],
                         post_weight=s["post_weight"], residual_scale=c["residual_scale"],
                         amax=s["amax"])
    return r, h, _bf16_of(s["amax"])


def _own_rotary(s):
    import nvfp4_block_scaled_05_amd as nv
    return nv.rotary(s["q"], s["positions"], s["plan"], k=s["k"], layout=s["case"]["layout"],
                     q_weight=s["q_weight"], k_weight=s["k_weight"])


def _own_attn(s):
    import nvfp4_block_scaled_05_amd as nv
    return nv.cross_attention(s["q"], s["k"], s["v"], kv_lengths=s["lengths"], key_mask=s["mask"])


def _own_lora(s):
    import nvfp4_block_scaled_05_amd as nv
    y = nv.lora_add(s["y"], s["x"], s["down"], s["up"], s["ids"], scales=s["scales"],
                    epilogue=s["case"]["epilogue"], y_amax=s["amax"], out=torch.empty_like(s["y"]))
    return y, _bf16_of(s["amax"])


def _plain_normalise(z, kind, weight, bias):
    if kind == "layer":
        z = z - z.mean(-1, keepdim=True)
    z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6)
    if weight is not None:
        z = z * weight
    return z if bias is None else z + bias


def _plain_norm(s):
    c = s["case"]
    z = s["y"].float()
    if c["post"] != "none":
        z = _plain_normalise(z, c["post"], s["post_weight"], None)
    if s["gate"] is not None:
        z = s["gate"].float()[:, None] * z
    r = c["residual_scale"] * s["x"].float() + z
    h = _plain_normalise(r, c["norm"], s["weight"], s["bias"])
    if s["scale"] is not None:
        h = h * (1 + s["scale"].float()[:, None]) + s["shift"].float()[:, None]
    h = h.to(BF16)
    return r.to(s["x"].dtype), h, h.abs().max().reshape(1) if c["amax"] else None


def _plain_rotary(s):
    c = s["case"]
    rot, pairs = c["rotary_dim"], c["rotary_dim"] // 2
    p = s["positions"] if s["positions"].dim() == 3 else s["positions"][..., None]
    angle = (p.double()[..., s["axis"]] * s["freq"])[:, :, None]
    cos = (angle.cos() * s["magnitude"]).float()
    sin = (angle.sin() * s["magnitude"]).float()
    outs = []
    for z, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        z = z.float()
        if w is not None:
            z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * w
        if c["layout"] == "half":
            a, b = z[..., :pairs], z[..., pairs:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = z[..., 0:rot:2], z[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        outs.append(torch.cat([turned, z[..., rot:]], -1).to(BF16))
    return tuple(outs)


def _plain_attn(s):
    c = s["case"]
    group = c["heads"] // c["kv_heads"]
    visible = torch.ones((c["batch"], c["keys"]), dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        visible = visible & (torch.arange(c["keys"], device="cuda") < s["lengths"][:, None])
    if s["mask"] is not None:
        visible = visible & s["mask"]
    zero = torch.zeros((), device="cuda")
    k = torch.where(visible[:, :, None, None], s["k"].float(), zero)
    v = torch.where(visible[:, :, None, None], s["v"].float(), zero)
    k = k.permute(0, 2, 3, 1).repeat_interleave(group, 1).contiguous()   # [B, H, D, keys]
    v = v.permute(0, 2, 1, 3).repeat_interleave(group, 1).contiguous()   # [B, H, keys, D]
    q = s["q"].float().permute(0, 2, 1, 3).contiguous() * c["dim"] ** -0.5
    sc = torch.matmul(q, k).masked_fill_(~visible[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    e = sc.sub_(torch.where(top.isinf(), zero, top)).exp_()
    o = torch.matmul(e, v) / e.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.permute(0, 2, 1, 3).to(BF16).contiguous()


def _plain_lora(s):
    c = s["case"]
    m, r = c["adapters"], c["rank"]
    t = s["x"].float() @ s["down"].float().reshape(m * r, -1).t()
    mine = s["ids"][:, None] == torch.arange(m, device="cuda")
    factor = torch.where(mine, s["scales"], torch.zeros((), device="cuda"))
    t = (t.view(-1, m, r) * factor[..., None]).view(-1, m * r)
    y = s["y"].float() + t @ s["up"].float().permute(1, 0, 2).reshape(-1, m * r).t()
    if c["epilogue"] == "gelu":
        y = 0.5 * y * torch.erfc(y * -(0.5 ** 0.5))
    y = y.to(BF16)
    return y, y.abs().max().reshape(1) if c["amax"] else None


_OWN = {"norm": _own_norm, "rotary": _own_rotary, "attn": _own_attn, "lora": _own_lora}
_PLAIN = {"norm": _plain_norm, "rotary": _plain_rotary, "attn": _plain_attn, "lora": _plain_lora}


# ----------------------------------------------------------------- bytes, flops

def work(case):
    c = case
    if c["op"] == "norm":
        n = c["batch"] * c["tokens"] * c["channels"]
        stream = 2 if c["stream"] == "bf16" else 4
        vectors = (3 * 2 * c["batch"] * c["channels"] if c["modulated"] else 0) + (
            2 * 4 * c["channels"] if c["weights"] else 0)
        return {"bytes": n * (2 * stream + 2 + 2) + vectors,
                "flops": n * (12 + (5 if c["post"] != "none" else 0))}
    if c["op"] == "rotary":
        tokens = c["batch"] * c["tokens"]
        n = tokens * (c["heads"] + c["kv_heads"]) * c["dim"]
        axes = len(_numbers(c["axes"])) or 1
        return {"bytes": 4 * n + 4 * tokens * axes + 6 * c["rotary_dim"],
                "flops": n * (3 * c["rotary_dim"] // c["dim"] + (4 if c["norm"] else 0)) or 1}
    if c["op"] == "attn":
        # keys a request sees: those of its length, thinned by the mask
        seen = sum(n * c["keep"] for n in _lengths(c))
        q = c["batch"] * c["queries"] * c["heads"] * c["dim"]
        return {"bytes": int(4 * q + 4 * seen * c["kv_heads"] * c["dim"]),
                "flops": int(4 * seen * c["queries"] * c["heads"] * c["dim"]) or 1}
    t, k, n, r = c["rows"], c["inner"], c["outer"], c["rank"]
    used = min(c["adapters"], c["requests"])
    return {"bytes": 2 * t * (k + 2 * n) + 2 * used * r * (k + n) + 4 * t,
            "flops": 2 * t * r * (k + n)}


# ------------------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _exact_norm(c, s):
    def norm(z, kind, weight, bias):
        mu = z.sum(-1, keepdim=True) / z.shape[-1] if kind == "layer" else 0.0
        var = ((z - mu) ** 2).sum(-1, keepdim=True) / z.shape[-1]
        z = (z - mu) / (var + 1e-6).sqrt()
        z = z if weight is None else z * weight.double()
        return z if bias is None else z + bias.double()

    rs, hs = [], []
    for b in range(c["batch"]):
        y = s["y"][b].double()
        y = y if c["post"] == "none" else norm(y, c["post"], s["post_weight"], None)
        r = c["residual_scale"] * s["x"][b].double() + (y if s["gate"] is None else s["gate"][b].double() * y)
        h = norm(r, c["norm"], s["weight"], s["bias"])
        if s["scale"] is not None:
            h = h * (1.0 + s["scale"][b].double()) + s["shift"][b].double()
        rs.append(r)
        hs.append(h)
    h = torch.stack(hs)
    return torch.stack(rs), h, h.abs().amax().reshape(1) if c["amax"] else None


def _exact_rotary(c, s):
    rot = c["rotary_dim"]
    p = s["positions"].reshape(c["batch"], c["tokens"], -1).double()
    freq, axis, magnitude = _frequencies(c)
    outs = []
    for z, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        z = z.double()
        if w is not None:
            z = z / ((z ** 2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt() * w.double()
        out = z.clone()
        for j in range(rot // 2):
            i0, i1 = (j, j + rot // 2) if c["layout"] == "half" else (2 * j, 2 * j + 1)
            a = (p[..., axis[j]] * freq[j])[..., None]
            out[..., i0] = magnitude * (z[..., i0] * a.cos() - z[..., i1] * a.sin())
            out[..., i1] = magnitude * (z[..., i0] * a.sin() + z[..., i1] * a.cos())
        outs.append(out)
    return tuple(outs)


def _exact_attn(c, s):
    out = torch.zeros((c["batch"], c["queries"], c["heads"], c["dim"]), dtype=F64, device="cuda")
    lengths = _lengths(c)
    for b in range(c["batch"]):
        kept = torch.arange(lengths[b], device="cuda")
        if s["mask"] is not None:
            kept = kept[s["mask"][b, :lengths[b]]]
        if kept.numel() == 0:
            continue
        for h in range(c["heads"]):
            hk = h * c["kv_heads"] // c["heads"]
            k, v = s["k"][b, kept, hk].double(), s["v"][b, kept, hk].double()
            w = torch.softmax(s["q"][b, :, h].double() @ k.t() / math.sqrt(c["dim"]), -1)
            out[b, :, h] = w @ v
    return out


def _exact_lora(c, s):
    y = s["y"].double()
    for a in range(c["adapters"]):
        rows = (s["ids"] == a).nonzero()[:, 0]
        if rows.numel():
            t = s["x"][rows].double() @ s["down"][a].double().t()
            y[rows] += s["scales"][a].double() * (t @ s["up"][a].double().t())
    if c["epilogue"] == "gelu":
        y = y / 2 * torch.special.erfc(-y / math.sqrt(2.0))
    return y, y.abs().amax().reshape(1) if c["amax"] else None


_EXACT = {"norm": _exact_norm, "rotary": _exact_rotary, "attn": _exact_attn, "lora": _exact_lora}
