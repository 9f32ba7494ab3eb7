"""Cases, plain forms and exact values of the operators around the attention kernels: rotary positions with per-head norms
(forward and backward), writing new tokens into a paged key/value cache, copying its pages, and decoding over it.

`run` computes a case in elementary torch operations, in 32 bits (angles and long sums in 64), rounded once at the end, or,
where `own` is true, by the package's entry points. `exact` gives the same values from the definitions in 64 bits."""
import math

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_EPS = 1e-6


# ---------------------------------------------------------------------------------------------------- the cases
def _rope(name, B, Hq, Hkv, L, d, rotary, dtype, interleaved=False, norm=False, backward=False, first=0, stretch=1.0, rows_first=True):
    """Queries [B, Hq, L, d] and keys [B, Hkv, L, d] at positions first + 0 .. L - 1; `rows_first`: they lie in memory as the
    projections give them, [B, L, H, d]. `stretch`: the context is that many times the trained one."""
    return {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hkv": Hkv, "L": L, "d": d, "rotary": rotary, "dtype": dtype, "interleaved": interleaved,
            "norm": norm, "backward": backward, "first": first, "stretch": stretch, "rows_first": rows_first}


def _append(name, B, Hq, Hkv, L, d, page, dtype, rotary=0, norm=False, ragged=False, cached=0):
    """Up to L new tokens for each of B sequences (`ragged`: 1 .. L of them, spread evenly) behind up to `cached` old ones.
    rotary > 0: queries and keys are rotated (and normalised) in the same call."""
    return {"name": name, "op": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "L": L, "d": d, "page": page, "dtype": dtype, "rotary": rotary, "norm": norm,
            "ragged": ragged, "cached": cached}


def _copy(name, pairs, Hkv, page, d, dtype):
    """`pairs` pages of keys and of values copied to free pages of the same cache."""
    return {"name": name, "op": "copy", "pairs": pairs, "Hkv": Hkv, "page": page, "d": d, "dtype": dtype}


def _decode(name, B, Hq, Hkv, shortest, longest, d, page, dtype, slots_first=False):
    """One query row for each of B sequences of `shortest` .. `longest` cached tokens, spread evenly; `slots_first`: a page
    lies in memory as [page, Hkv, d] and not as [Hkv, page, d]."""
    return {"name": name, "op": "decode", "B": B, "Hq": Hq, "Hkv": Hkv, "shortest": shortest, "longest": longest, "d": d, "page": page, "dtype": dtype,
            "slots_first": slots_first}


def listed():
    return [
        # One decoding step of eight sequences: latency counts.
        _rope("rope step", 8, 32, 8, 1, 128, 128, "bf16", norm=True, first=8191),
        # A training step's queries and keys on their way into the causal forward pass of 8 x 32 x 512 x 128.
        _rope("rope training", 8, 32, 32, 512, 128, 128, "fp16"),
        # The way back through norms and rotation, with the norms' weight gradients; queries share keys' heads four to one.
        _rope("rope norm backward", 4, 32, 8, 2048, 128, 128, "bf16", norm=True, backward=True),
        # Half of a short head, interleaved pairs, an odd length at far positions of a stretched context.
        _rope("rope far part", 1, 16, 16, 100003, 64, 32, "fp16", interleaved=True, first=900000, stretch=32.0, rows_first=False),
        # One decoding step's keys and values of 64 sequences into their pages, norms and rotation in the same call.
        _append("append step", 64, 32, 8, 1, 128, 16, "bf16", rotary=128, norm=True, cached=8191),
        # Eight prompts of a padded batch.
        _append("append prompts", 8, 32, 8, 2048, 128, 16, "fp16", rotary=128, ragged=True, cached=300),
        # The last pages of seven sequences that are forked.
        _copy("copy fork", 7, 8, 16, 128, "fp16"),
        # A cache that is compacted.
        _copy("copy compact", 4000, 8, 16, 128, "bf16"),
        # A single short sequence: latency counts.
        _decode("decode one", 1, 8, 8, 1000, 1000, 128, 16, "fp16"),
        # The batched decoding step of 8 x 32 heads x 8192 keys, paged.
        _decode("decode batch", 8, 32, 32, 8192, 8192, 128, 64, "fp16"),
        # Sequences of very different lengths, one of them empty, four query heads to a key head.
        _decode("decode ragged", 64, 32, 8, 0, 16000, 128, 16, "bf16", slots_first=True),
        # The longest sequence, 1,048,576 tokens.
        _decode("decode long", 1, 32, 8, 1048576, 1048576, 128, 128, "bf16"),
    ]


def _spread(rng, low, high):
    """A whole number of low .. high, evenly over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "copy", "decode", "decode"])
    dtype, d, Hkv, group = rng.choice(["fp16", "bf16"]), rng.choice([64, 128, 128, 256, 512]), rng.choice([1, 2, 5, 8, 16, 32]), rng.choice([1, 1, 2, 4, 7, 8, 16])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128, 256])
    if op == "rope":
        B = _spread(rng, 1, 64)
        L = _spread(rng, 1, max(1, int(1.5e8 / (B * Hkv * (group + 1) * d))))
        case = _rope("", B, Hkv * group, Hkv, L, d, rng.choice([d, d, d // 2, d // 4]), dtype, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5,
                     _spread(rng, 1, 2000000) - 1, rng.choice([1.0, 4.0, 32.0]), rng.random() < 0.5)
    elif op == "append":
        B = _spread(rng, 1, 128)
        L = _spread(rng, 1, max(1, int(6e7 / (B * Hkv * (group + 2) * d))))
        case = _append("", B, Hkv * group, Hkv, L, d, page, dtype, rng.choice([0, d, d, d // 2]), rng.random() < 0.5, rng.random() < 0.5,
                       rng.choice([0, _spread(rng, 1, max(1, int(1e8 / (B * Hkv * d))))]))
        case["norm"] = case["norm"] and case["rotary"] > 0
    elif op == "copy":
        case = _copy("", _spread(rng, 1, max(1, min(6000, int(2e8 / (Hkv * page * d))))), Hkv, page, d, dtype)
    else:
        B = _spread(rng, 1, 200)
        longest = _spread(rng, 1, max(1, min(1048576, int(5e8 / (B * Hkv * d)))))
        case = _decode("", B, Hkv * group, Hkv, rng.choice([0, 1, longest, longest // 2]), longest, d, page, dtype, rng.random() < 0.5)
    del case["name"]
    return case


def _lengths(case):
    """Tokens of each sequence of a decode case; old and new tokens of each sequence of an append case."""
    B = case["B"]
    if case["op"] == "decode":
        return [case["shortest"] + (case["longest"] - case["shortest"]) * b // max(1, B - 1) if B > 1 else case["longest"] for b in range(B)]
    old = [case["cached"] - case["cached"] * b // (2 * B) for b in range(B)]
    new = [1 + (case["L"] - 1) * b // max(1, B - 1) if case["ragged"] and B > 1 else case["L"] for b in range(B)]
    return old, new


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["B"] * case["L"] * (case["Hq"] + case["Hkv"]) * d
        return {"bytes": n * (6 if case["backward"] and case["norm"] else 4), "flops": n * (3 + (8 if case["backward"] else 4) * case["norm"])}
    if case["op"] == "append":
        rows, all_rows = sum(_lengths(case)[1]), case["B"] * case["L"]
        n = rows * 2 * case["Hkv"] * d + (rows + all_rows) // 2 * case["Hq"] * d * (case["rotary"] > 0)
        return {"bytes": n * 4, "flops": n * (3 + 4 * case["norm"]) * (case["rotary"] > 0)}
    if case["op"] == "copy":
        return {"bytes": case["pairs"] * case["Hkv"] * case["page"] * d * 8, "flops": 0}
    keys = sum(_lengths(case))
    return {"bytes": keys * case["Hkv"] * d * 4 + case["B"] * case["Hq"] * (d * 4 + 4), "flops": 4 * keys * case["Hq"] * d}


# ---------------------------------------------------------------------------------------------------- inputs
def _heads(g, dt, B, H, L, d, rows_first, sigma=1.0):
    if rows_first:
        return (torch.randn(B, L, H, d, generator=g, device="cuda", dtype=dt) * sigma).transpose(1, 2)
    return torch.randn(B, H, L, d, generator=g, device="cuda", dtype=dt) * sigma


def _frequencies(rotary, stretch):
    """inv_freq[i] = 10000^(-2i / rotary), slowed by `stretch`, and the factor on cosine and sine that goes with it."""
    i = torch.arange(rotary // 2, dtype=torch.float64, device="cuda")
    return torch.pow(10000.0, -2.0 * i / rotary) / stretch, 1.0 + 0.1 * math.log(stretch)


def _tables(g, pages, page, lengths, longest):
    """Page tables [B, width] of sequences of `lengths` tokens, the pages dealt at random, -1 behind a sequence's last page."""
    width = max(1, -(-longest // page))
    need = torch.tensor([-(-n // page) for n in lengths], device="cuda")
    used = torch.arange(width, device="cuda")[None] < need[:, None]
    place = (torch.cumsum(need, 0) - need)[:, None] + torch.arange(width, device="cuda")[None]
    deal = torch.randperm(pages, generator=g, device="cuda")
    return torch.where(used, deal[place.clamp(max=pages - 1)], -1).to(torch.int32)


def _cache(g, dt, pages, Hkv, page, d, slots_first=False):
    if slots_first:
        return [torch.randn(pages, page, Hkv, d, generator=g, device="cuda", dtype=dt).transpose(1, 2) for _ in range(2)]
    return [torch.randn(pages, Hkv, page, d, generator=g, device="cuda", dtype=dt) for _ in range(2)]


def _weights(g, dt, d):
    return [(1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt) for _ in range(2)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d = _TYPES[case["dtype"]], case["d"]
    s = dict(case)
    if case["op"] == "rope":
        B, L = case["B"], case["L"]
        s["q"], s["k"] = (_heads(g, dt, B, H, L, d, case["rows_first"]) for H in (case["Hq"], case["Hkv"]))
        if case["backward"]:
            s["dq"], s["dk"] = (_heads(g, dt, B, H, L, d, False) for H in (case["Hq"], case["Hkv"]))
        s["positions"] = (case["first"] + torch.arange(L, device="cuda", dtype=torch.int32)[None].expand(B, L)).contiguous()
        s["inv_freq"], s["factor"] = _frequencies(case["rotary"], case["stretch"])
        s["wq"], s["wk"] = _weights(g, dt, d) if case["norm"] else (None, None)
    elif case["op"] == "append":
        B, L, Hkv, page = case["B"], case["L"], case["Hkv"], case["page"]
        old, new = _lengths(case)
        after = [a + n for a, n in zip(old, new)]
        pages = sum(-(-n // page) for n in after) + 3
        s["table"] = _tables(g, pages, page, after, max(after))
        s["lengths"] = torch.tensor(after, device="cuda", dtype=torch.int32)
        s["counts"] = torch.tensor(new, device="cuda", dtype=torch.int32)
        s["k_pages"], s["v_pages"] = _cache(g, dt, pages, Hkv, page, d)
        # Queries, keys and values are parts of one projection's output.
        qkv = torch.randn(B, L, case["Hq"] + 2 * Hkv, d, generator=g, device="cuda", dtype=dt).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv.split([case["Hq"], Hkv, Hkv], dim=1)
        s["wq"], s["wk"] = _weights(g, dt, d) if case["norm"] else (None, None)
        s["inv_freq"], s["factor"] = _frequencies(case["rotary"], 1.0) if case["rotary"] else (None, 1.0)
    elif case["op"] == "copy":
        n = case["pairs"]
        pages = 2 * n + 5
        s["k_pages"], s["v_pages"] = _cache(g, dt, pages, case["Hkv"], case["page"], d)
        deal = torch.randperm(pages, generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
        s["src"], s["dst"] = deal[:n].contiguous(), deal[n:2 * n].contiguous()  # the page bookkeeping is on the host
    else:
        B, page = case["B"], case["page"]
        lengths = _lengths(case)
        order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
        lengths = [lengths[i] for i in order]
        pages = sum(-(-n // page) for n in lengths) + 3
        s["table"] = _tables(g, pages, page, lengths, case["longest"])
        s["lengths"] = torch.tensor(lengths, device="cuda", dtype=torch.int32)
        s["k_pages"], s["v_pages"] = _cache(g, dt, pages, case["Hkv"], page, d, case["slots_first"])
        s["q"] = torch.randn(B, case["Hq"], d, generator=g, device="cuda", dtype=dt)
    return s


# ---------------------------------------------------------------------------------------------------- the plain forms
def _turn(x, positions, inv_freq, factor, interleaved):
    """The first 2 len(inv_freq) elements of each head turned in pairs by positions x inv_freq, in the type of x."""
    angle = positions.double()[..., None] * inv_freq  # [B, L, rotary / 2]
    c, s = ((factor * f(angle)).to(x.dtype)[:, None] for f in (torch.cos, torch.sin))
    rotary = 2 * inv_freq.numel()
    r, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)
    a, b = r[..., :rotary // 2], r[..., rotary // 2:]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1)


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * w.to(x.dtype)


def _plain_rope(x, w, s):
    y = x.float()
    y = y if w is None else _norm(y, w)
    return _turn(y, s["positions"], s["inv_freq"], s["factor"], s["interleaved"]).to(x.dtype).contiguous()


def _plain_rope_back(dz, x, w, s):
    dy = _turn(dz.float(), -s["positions"], s["inv_freq"], s["factor"], s["interleaved"])
    if w is None:
        return dy.to(dz.dtype).contiguous(), None
    y = x.float()
    rstd = torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS)
    y = y * rstd
    dw = (dy * y).sum((0, 1, 2), dtype=torch.float64).float()
    g = dy * w.float()
    return (rstd * (g - y * (g * y).mean(-1, keepdim=True))).to(dz.dtype).contiguous(), dw


def _plain_append(s):
    B, L = s["B"], s["L"]
    t = torch.arange(L, device="cuda")[None].expand(B, L)
    there = t < s["counts"][:, None]
    pos = s["lengths"][:, None] - s["counts"][:, None] + t
    k, v, q = s["k"], s["v"], None
    if s["rotary"]:
        at = {"positions": pos, "inv_freq": s["inv_freq"], "factor": s["factor"], "interleaved": False}
        k = _plain_rope(k, s["wk"], at)
        q = torch.where(there[:, None, :, None], _plain_rope(s["q"], s["wq"], at), 0)
    t = torch.minimum(t, s["counts"][:, None] - 1).long()  # rows behind the last one write what that one writes
    pos = (s["lengths"][:, None] - s["counts"][:, None] + t).long()
    page, slot = torch.gather(s["table"].long(), 1, pos // s["page"]), pos % s["page"]
    b = torch.arange(B, device="cuda")[:, None].expand(B, L)
    s["k_pages"][page, :, slot] = k[b, :, t]
    s["v_pages"][page, :, slot] = v[b, :, t]
    return [s["k_pages"], s["v_pages"]] + ([] if q is None else [q])


def _plain_decode(s):
    B, Hkv, d = s["B"], s["Hkv"], s["d"]

    def sequences(pages):  # [B, Hkv, keys, d]
        return pages[s["table"].clamp(min=0).long()].transpose(1, 2).reshape(B, Hkv, -1, d).float()

    k = sequences(s["k_pages"])
    x = (s["q"].float().view(B, Hkv, -1, d) @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    x = torch.where(torch.arange(x.shape[3], device="cuda") < s["lengths"][:, None, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0))
    total = p.sum(-1, keepdim=True)
    o = (p @ sequences(s["v_pages"])) / torch.where(total > 0, total, 1)
    return [o.to(s["q"].dtype).view(B, -1, d), (top + torch.log(total)).view(B, -1)]


def run(state):
    s = state
    if own:
        import scaled_dot_product_sdpa_gb300 as gb
        if s["op"] == "rope":
            if not s["backward"]:
                return gb.attn_rope(s["q"], s["k"], s["inv_freq"], positions=s["positions"], interleaved=s["interleaved"], factor=s["factor"],
                                    q_weight=s["wq"], k_weight=s["wk"], eps=_EPS)
            if not s["norm"]:
                return gb.attn_rope_bwd(s["dq"], s["dk"], s["inv_freq"], positions=s["positions"], interleaved=s["interleaved"], factor=s["factor"])
            return gb.attn_rope_bwd(s["dq"], s["dk"], s["inv_freq"], positions=s["positions"], interleaved=s["interleaved"], factor=s["factor"],
                                    q=s["q"], k=s["k"], q_weight=s["wq"], k_weight=s["wk"], eps=_EPS)
        if s["op"] == "append":
            if not s["rotary"]:
                gb.attn_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], counts=s["counts"])
                return [s["k_pages"], s["v_pages"]]
            q = gb.attn_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], counts=s["counts"], q=s["q"], inv_freq=s["inv_freq"],
                                     factor=s["factor"], q_weight=s["wq"], k_weight=s["wk"], eps=_EPS)
            return [s["k_pages"], s["v_pages"], q]
        if s["op"] == "copy":
            gb.attn_cache_copy(s["k_pages"], s["v_pages"], s["src"], s["dst"])
            return [s["k_pages"], s["v_pages"]]
        return gb.attn_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"])
    if s["op"] == "rope":
        if not s["backward"]:
            return [_plain_rope(s["q"], s["wq"], s), _plain_rope(s["k"], s["wk"], s)]
        (dq, dwq), (dk, dwk) = _plain_rope_back(s["dq"], s["q"], s["wq"], s), _plain_rope_back(s["dk"], s["k"], s["wk"], s)
        return [dq, dk] if dwq is None else [dq, dk, dwq, dwk]
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "copy":
        src, dst = s["src"].cuda().long(), s["dst"].cuda().long()
        s["k_pages"][dst] = s["k_pages"][src]
        s["v_pages"][dst] = s["v_pages"][src]
        return [s["k_pages"], s["v_pages"]]
    return _plain_decode(s)


# ---------------------------------------------------------------------------------------------------- in 64 bits
def _exact_rope(x, w, positions, inv_freq, factor, interleaved):
    """A pair as a complex number times factor e^(i angle), after the norm."""
    y = x.double()
    if w is not None:
        y = y / ((y * y).sum(-1, keepdim=True) / y.shape[-1] + _EPS).sqrt() * w.double()
    n = inv_freq.numel()
    i = torch.arange(n, device="cuda")
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    angle = positions.double()[:, None, :, None] * inv_freq
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.full_like(angle, factor), angle)
    out = y.clone(memory_format=torch.contiguous_format)
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rope_back(dz, x, w, s):
    """Through torch's own differentiation of the forward definition."""
    x = x.double().contiguous().requires_grad_(True)
    w = None if w is None else w.double().requires_grad_(True)
    y = x if w is None else x / ((x * x).mean(-1, keepdim=True) + _EPS).sqrt() * w
    n = s["inv_freq"].numel()
    i = torch.arange(n, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + n)
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"]
    c, t = s["factor"] * angle.cos(), s["factor"] * angle.sin()
    g = dz.double()
    value = ((y[..., first] * c - y[..., second] * t) * g[..., first]).sum() + ((y[..., second] * c + y[..., first] * t) * g[..., second]).sum()
    value = value + (y[..., 2 * n:] * g[..., 2 * n:]).sum()
    return torch.autograd.grad(value, [x] if w is None else [x, w])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        if not case["backward"]:
            return [_exact_rope(s[x], s["w" + x], s["positions"], s["inv_freq"], s["factor"], s["interleaved"]) for x in "qk"]
        q, k = (_exact_rope_back(s["d" + x], s[x], s["w" + x], s) for x in "qk")
        return [q[0], k[0]] if len(q) == 1 else [q[0], k[0], q[1], k[1]]
    if case["op"] == "copy":
        src, dst = s["src"].tolist(), s["dst"].tolist()
        for pages in (s["k_pages"], s["v_pages"]):
            for a in range(0, len(src), 512):
                pages.index_copy_(0, torch.tensor(dst[a:a + 512], device="cuda"), pages.index_select(0, torch.tensor(src[a:a + 512], device="cuda")))
        return [s["k_pages"].double(), s["v_pages"].double()]
    lengths, table = s["lengths"].tolist(), s["table"].tolist()
    if case["op"] == "append":
        counts = s["counts"].tolist()
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        k, v, q = s["k"].double(), s["v"], None
        if case["rotary"]:
            pos = torch.tensor([[n - c + t for t in range(case["L"])] for n, c in zip(lengths, counts)], device="cuda")
            k, q = (_exact_rope(s[x], s["w" + x], pos, s["inv_freq"], s["factor"], False) for x in "kq")
        for b, (n, c) in enumerate(zip(lengths, counts)):
            at = range(n - c, n)
            page = torch.tensor([table[b][p // case["page"]] for p in at], device="cuda")
            slot = torch.tensor([p % case["page"] for p in at], device="cuda")
            k_pages[page, :, slot] = k[b, :, :c].transpose(0, 1)
            v_pages[page, :, slot] = v[b, :, :c].transpose(0, 1).double()
            if q is not None:
                q[b, :, c:] = 0
        return [k_pages, v_pages] if q is None else [k_pages, v_pages, q]
    G = case["Hq"] // case["Hkv"]
    o = torch.zeros(case["B"], case["Hq"], case["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths):
        if n == 0:
            continue
        at = s["table"][b, :-(-n // case["page"])].long()
        for h in range(case["Hkv"]):
            k, v = (x[at, h].reshape(-1, case["d"])[:n].double() for x in (s["k_pages"], s["v_pages"]))
            x = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(case["d"])
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            o[b, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return [o, lse]
