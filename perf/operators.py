"""The operators of the quantised history cache, as cases to be timed and compared.

Rotary positions (forward and backward), quantising keys and values as they are written
into history pages, reading selected pages back into the contiguous active cache, and
attention of a few query tokens straight over the quantised pages.  ``run`` computes a
case in elementary torch operations, or through the package where ``own`` is true;
``exact`` computes it once more in 64 bits.

A page of P rows, H heads of d columns is one block of bytes: the codes [P][H][d] (8 or
4 bits each; of two 4-bit codes in a byte the even column is the low one), then, from the
next multiple of 256 bytes, fp32 scales [P][H][d / group]; its size is a multiple of 1024.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
QMAX = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}
TINY = 2.0 ** -100  # a group whose largest magnitude is below this is stored as zeros


def listed():
    return [
        # one new token's queries and keys of a 14B layer (40 heads): the launch is what counts
        dict(name="rope_token", kind="rope", T=1, Hq=40, Hk=40, d=128, rot=128, layout="interleaved", axes=3, dtype="bf16",
             scaling="none", far=1 << 14, strided=False),
        # the queries and keys of a 720p chunk (3 latent frames of 3600 tokens), rotated by frame, row and column
        dict(name="rope_chunk_720p", kind="rope", T=10800, Hq=40, Hk=40, d=128, rot=128, layout="interleaved", axes=3,
             dtype="bf16", scaling="none", far=1, strided=False),
        # part of a narrow head in the half layout, stretched for a long context, far positions, fp32, rows inside a fused projection
        dict(name="rope_part_fp32", kind="rope", T=4099, Hq=12, Hk=3, d=64, rot=32, layout="half", axes=1, dtype="fp32",
             scaling="yarn", far=1 << 20, strided=True),
        # gradients of a 480p chunk of the 1.3B layer (12 heads)
        dict(name="rope_bwd_480p", kind="rope_bwd", T=4680, Hq=12, Hk=12, d=128, rot=128, layout="interleaved", axes=3,
             dtype="bf16", scaling="none", far=1, strided=False),
        # gradients with an odd token count and shared keys, half layout, fp16
        dict(name="rope_bwd_half_fp16", kind="rope_bwd", T=7777, Hq=40, Hk=5, d=128, rot=128, layout="half", axes=1, dtype="fp16",
             scaling="ntk", far=1 << 16, strided=False),
        # one token appended to the open page: latency
        dict(name="write_token", kind="write", T=1, first=201, P=256, NP=2, H=40, d=128, fmt="e4m3", group=128, dtype="bf16",
             rot=0, layout="half", axes=1),
        # a whole 480p page (8 latent frames of 1560 tokens) of the 14B layer sealed, its keys rotated on the way
        dict(name="write_page_480p", kind="write", T=12480, first=0, P=12480, NP=1, H=40, d=128, fmt="e4m3", group=128,
             dtype="bf16", rot=128, layout="interleaved", axes=3),
        # an odd run of fp32 rows across several small pages, narrow heads, a scale for every 32 columns, 8-bit integers
        dict(name="write_run_int8", kind="write", T=1563, first=77, P=200, NP=9, H=12, d=64, fmt="int8", group=32, dtype="fp32",
             rot=0, layout="half", axes=1),
        # the active cache of the 14B layer at 480p: 4 pages, keys rotated to their places in the active cache
        dict(name="read_480p", kind="read", Kp=4, P=12480, NP=6, H=40, d=128, fmt="e4m3", group=128, rot=128, layout="interleaved",
             axes=3, means=True),
        # three odd pages in 4 bits, part of the head rotated in the half layout
        dict(name="read_odd_int4", kind="read", Kp=3, P=1563, NP=5, H=12, d=128, fmt="int4", group=32, rot=64, layout="half",
             axes=1, means=False),
        # one token over four 480p pages of the 1.3B layer
        dict(name="attn_token", kind="attn", T=1, g=1, Kp=4, P=12480, NP=4, n=49920, H=12, d=128, fmt="e4m3", group=128, out="fp32"),
        # a few tokens of shared-key heads over odd pages, the last one partly filled, 8-bit integers
        dict(name="attn_few_int8", kind="attn", T=5, g=3, Kp=4, P=12345, NP=6, n=41234, H=40, d=64, fmt="int8", group=32, out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "rope_bwd", "write", "read", "attn"])
    d = rng.choice([64, 128])
    layout = rng.choice(["interleaved", "half"])
    axes = rng.choice([1, 3])
    if kind in ("rope", "rope_bwd"):
        Hk = _log(rng, 1, 40)
        return dict(kind=kind, T=_log(rng, 1, 10800), Hq=min(40, Hk * rng.choice([1, 1, 2, 4])), Hk=Hk, d=d,
                    rot=rng.choice([d, d, d // 2, 48]), layout=layout, axes=axes, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), far=_log(rng, 1, 1 << 20), strided=rng.random() < 0.3)
    if kind == "write":
        T, P = _log(rng, 1, 12480), _log(rng, 16, 12480)
        first = rng.randrange(P)
        fmt = rng.choice(["e4m3", "int8"])
        # codes of whole numbers have to be equal: those are written as they come, unrotated
        rot = rng.choice([0, d, d // 2]) if fmt == "e4m3" else 0
        return dict(kind=kind, T=T, first=first, P=P, NP=-(-(first + T) // P), H=_log(rng, 1, 40), d=d, fmt=fmt,
                    group=rng.choice([g for g in (32, 64, 128) if g <= d]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    rot=rot, layout=layout, axes=axes)
    fmt = rng.choice(["e4m3", "int8", "int4"])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    Kp, P, H = rng.randrange(1, 5), _log(rng, 16, 12480), _log(rng, 1, 40)
    NP = Kp + rng.randrange(0, 3)
    if kind == "read":
        return dict(kind=kind, Kp=Kp, P=P, NP=NP, H=H, d=d, fmt=fmt, group=group, rot=rng.choice([0, d, d, d // 2]), layout=layout,
                    axes=axes, means=rng.random() < 0.5)
    g = rng.choice([1, 1, 2, 5])
    return dict(kind=kind, T=_log(rng, 1, max(1, 16 // g)), g=g, Kp=Kp, P=P, NP=NP, n=rng.randrange((Kp - 1) * P + 1, Kp * P + 1), H=H, d=d,
                fmt=fmt, group=group, out=rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------ sizes

def _axis_pairs(rot, axes):
    """Pairs of each axis: all of them, or frame / row / column with what is left over going to the frame axis."""
    pairs = rot // 2
    return [pairs] if axes == 1 else [pairs - 2 * (pairs // 3), pairs // 3, pairs // 3]


def _code_bytes(c):
    return c["P"] * c["H"] * c["d"] * (1 if c["fmt"] != "int4" else 0.5)


def _page(c):
    """(byte offset of the scales, bytes of the page)"""
    off = -(-int(_code_bytes(c)) // 256) * 256
    return off, -(-(off + 4 * c["P"] * c["H"] * (c["d"] // c["group"])) // 1024) * 1024


def work(c):
    if c["kind"] in ("rope", "rope_bwd"):
        e = c["T"] * (c["Hq"] + c["Hk"])
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * e * c["d"] * size + 4 * c["T"] * c["axes"], "flops": 3 * e * c["rot"]}
    row = c["H"] * c["d"]
    coded = row * (1 if c["fmt"] != "int4" else 0.5) + 4 * row / c["group"]
    if c["kind"] == "write":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * c["T"] * (row * size + coded), "flops": c["T"] * (6 * row + 3 * c["H"] * c["rot"])}
    if c["kind"] == "read":
        n = c["Kp"] * c["P"]
        means = 4 * row * -(-n // 128) if c["means"] else 0
        return {"bytes": 2 * n * (coded + 2 * row) + means, "flops": n * (2 * row + 3 * c["H"] * c["rot"])}
    rows = c["T"] * c["g"] * c["H"]
    return {"bytes": 2 * c["n"] * coded + rows * c["d"] * (2 + (2 if c["out"] == "bf16" else 4)) + 4 * rows,
            "flops": 4 * rows * c["n"] * c["d"]}


# ------------------------------------------------------------------ inputs

def _frequencies(rot, axes, scaling):
    """(fp64 angle per position of every pair, factor on cos and sin): each axis has frequencies base^(-2i/dim) of
    its own; a long context divides them (linear), raises the base (ntk) or blends by wavelength (yarn)."""
    base, factor, context = 10000.0, 4.0, 4096
    parts = []
    for n in _axis_pairs(rot, axes):
        i, dim = torch.arange(n, dtype=torch.float64), 2 * n
        f = base ** (-2 * i / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "ntk" and dim > 2:
            f = (base * factor ** (dim / (dim - 2))) ** (-2 * i / dim)
        elif scaling == "yarn":
            turns = context * f / (2 * math.pi)
            keep = ((torch.log(turns) - math.log(1.0)) / (math.log(32.0) - math.log(1.0))).clamp(0, 1)
            f = f * keep + f / factor * (1 - keep)
        parts.append(f)
    return torch.cat(parts).cuda(), (0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0)


def _positions(n, axes, far, gen):
    """int32 [axes, n]: a running position from a place up to `far`, or frame, row and column of a latent video."""
    at = torch.arange(n, device="cuda", dtype=torch.int32)
    start = int(torch.randint(0, far, (1,), generator=gen, device="cuda"))
    if axes == 1:
        return (at + start)[None].contiguous()
    width, frame = 52, 1560  # a 480p latent frame: 30 rows of 52 tokens
    return torch.stack([at // frame + start, at % frame // width, at % width]).contiguous()


def _rotary(s, rot, axes, scaling, far, n, gen):
    s["inv_freq"], s["mscale"] = _frequencies(rot, axes, scaling)
    s["axis_pairs"] = _axis_pairs(rot, axes)
    s["axis_of_pair"] = torch.repeat_interleave(torch.arange(axes, device="cuda"), torch.tensor(s["axis_pairs"], device="cuda"))
    s["pos"] = _positions(n, axes, far, gen)


def _rows(T, H, d, dtype, strided, gen):
    if strided:  # the first H heads of a wider fused projection
        return torch.randn(T, 2 * H, d, generator=gen, device="cuda").to(dtype)[:, :H]
    return torch.randn(T, H, d, generator=gen, device="cuda").to(dtype)


def _encode(x, fmt, group):
    """Codes (uint8 [T, H, d], or two to a byte) and fp32 scales [T, H, d / group] of fp32 rows, by the elementwise definition."""
    q = x.unflatten(-1, (-1, group))
    amax = q.abs().amax(-1)
    kept = amax >= TINY
    scale = torch.where(kept, amax / QMAX[fmt], 0.0)
    inverse = torch.where(kept, QMAX[fmt] / amax, 0.0)
    q = (q * inverse[..., None]).flatten(-2)
    if fmt == "e4m3":
        return q.to(torch.float8_e4m3fn).view(torch.uint8), scale
    q = q.round().clamp(-QMAX[fmt], QMAX[fmt]).to(torch.int8).view(torch.uint8)
    if fmt == "int4":
        q = (q[..., 0::2] & 15) | (q[..., 1::2] << 4)
    return q, scale


def _code_view(pages, c):
    n = int(_code_bytes(c))
    return pages[:, :n].unflatten(1, (c["P"], c["H"], -1))


def _scale_view(pages, c):
    off, _ = _page(c)
    n = 4 * c["P"] * c["H"] * (c["d"] // c["group"])
    return pages[:, off:off + n].view(torch.float32).unflatten(1, (c["P"], c["H"], -1))


def _addresses(pages):
    step = pages.stride(0)
    return torch.arange(pages.shape[0], dtype=torch.int64, device="cuda") * step + pages.data_ptr()


def _filled_pages(c, gen, offset):
    """Pages of random rows; keys of one page share an offset, as the keys of one scene do."""
    pages = torch.zeros(c["NP"], _page(c)[1], dtype=torch.uint8, device="cuda")
    codes, scales = _code_view(pages, c), _scale_view(pages, c)
    for p in range(c["NP"]):
        x = torch.randn(c["P"], c["H"], c["d"], generator=gen, device="cuda")
        if offset:
            x += 0.5 * torch.randn(c["H"], c["d"], generator=gen, device="cuda")
        codes[p], scales[p] = _encode(x.bfloat16().float(), c["fmt"], c["group"])
    return pages


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": c}
    if c["kind"] in ("rope", "rope_bwd"):
        dt = DTYPES[c["dtype"]]
        s["q"], s["k"] = (_rows(c["T"], h, c["d"], dt, c["strided"], gen) for h in (c["Hq"], c["Hk"]))
        s["q_out"], s["k_out"] = (torch.empty(c["T"], h, c["d"], dtype=dt, device="cuda") for h in (c["Hq"], c["Hk"]))
        _rotary(s, c["rot"], c["axes"], c["scaling"], c["far"], c["T"], gen)
        return s
    if c["kind"] == "write":
        dt = DTYPES[c["dtype"]]
        s["k"], s["v"] = (_rows(c["T"], c["H"], c["d"], dt, False, gen) for _ in range(2))
        s["pages_k"], s["pages_v"] = (torch.zeros(c["NP"], _page(c)[1], dtype=torch.uint8, device="cuda") for _ in range(2))
        if c["rot"]:
            _rotary(s, c["rot"], c["axes"], "none", 4096, c["T"], gen)
    else:
        s["pages_k"], s["pages_v"] = _filled_pages(c, gen, True), _filled_pages(c, gen, False)
        s["sel"] = torch.randperm(c["NP"], generator=gen, device="cuda")[:c["Kp"]].sort().values.int()
        n = c["Kp"] * c["P"]
        if c["kind"] == "read":
            s["kc"], s["vc"] = (torch.empty(n, c["H"], c["d"], dtype=torch.bfloat16, device="cuda") for _ in range(2))
            s["means"] = torch.empty(-(-n // 128), c["H"], c["d"], device="cuda") if c["means"] else None
            if c["rot"]:
                _rotary(s, c["rot"], c["axes"], "none", 4096, n, gen)
        else:
            Hq = c["H"] * c["g"]
            s["q"] = torch.randn(c["T"], Hq, c["d"], generator=gen, device="cuda").bfloat16()
            s["out"] = torch.empty(c["T"], Hq, c["d"], dtype=DTYPES[c["out"]], device="cuda")
            s["lse"] = torch.empty(c["T"], Hq, device="cuda")
            s["n_rows"] = torch.tensor([c["n"]], dtype=torch.int32, device="cuda")
    s["table_k"], s["table_v"] = _addresses(s["pages_k"]), _addresses(s["pages_v"])
    return s


# ------------------------------------------------------------------ plain forms

def _rotate(x, s, sign=1.0):
    """Rotary positions on fp32 rows [T, H, d]: pair p of a row turns by pos * inv_freq[p]; angles in 64 bits."""
    c, rot = s["case"], s["case"]["rot"]
    angle = s["pos"][s["axis_of_pair"]].double().T * s["inv_freq"]
    cos, sin = ((f(angle) * s["mscale"]).float()[:, None] for f in (torch.cos, torch.sin))
    sin = sin * sign
    out = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2] = a * cos - b * sin
        out[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2] = a * cos - b * sin
        out[..., 1:rot:2] = b * cos + a * sin
    return out


def _decode(pages, s):
    """fp32 rows [Kp * P, H, d] of the selected pages."""
    c = s["case"]
    codes, scale = _code_view(pages, c)[s["sel"]], _scale_view(pages, c)[s["sel"]]
    if c["fmt"] == "e4m3":
        x = codes.view(torch.float8_e4m3fn).float()
    elif c["fmt"] == "int8":
        x = codes.view(torch.int8).float()
    else:
        x = torch.stack([(codes << 4).view(torch.int8) >> 4, codes.view(torch.int8) >> 4], -1).flatten(-2).float()
    return (x.unflatten(-1, (-1, c["group"])) * scale[..., None]).flatten(-2).flatten(0, 1)


def _code_values(pages, c):
    x = _code_view(pages, c)
    return x.view(torch.float8_e4m3fn if c["fmt"] == "e4m3" else torch.int8)


def _written(s):
    c = s["case"]
    return {"k": _code_values(s["pages_k"], c), "v": _code_values(s["pages_v"], c),
            "k_scale": _scale_view(s["pages_k"], c), "v_scale": _scale_view(s["pages_v"], c)}


def _block_means(x):
    """Means of 128-row blocks, the last one over the rows it has."""
    n = x.shape[0]
    pad = torch.zeros(-n % 128, *x.shape[1:], device=x.device, dtype=x.dtype)
    total = torch.cat([x, pad]).unflatten(0, (-1, 128)).sum(1)
    count = torch.full((total.shape[0], 1, 1), 128.0, device=x.device, dtype=x.dtype)
    count[-1] = n - 128 * (total.shape[0] - 1)
    return total / count


def _plain(s):
    c = s["case"]
    if c["kind"] in ("rope", "rope_bwd"):
        sign = -1.0 if c["kind"] == "rope_bwd" else 1.0
        return {n: _rotate(s[n].float(), s, sign).to(s[n].dtype) for n in ("q", "k")}
    if c["kind"] == "write":
        rows = torch.arange(c["first"], c["first"] + c["T"], device="cuda")
        at = (rows // c["P"], rows % c["P"])
        k = s["k"].float()
        k = _rotate(k, s) if c["rot"] else k
        ck, sk = _encode(k, c["fmt"], c["group"])
        cv, sv = _encode(s["v"].float(), c["fmt"], c["group"])
        _code_view(s["pages_k"], c)[at], _scale_view(s["pages_k"], c)[at] = ck, sk
        _code_view(s["pages_v"], c)[at], _scale_view(s["pages_v"], c)[at] = cv, sv
        return _written(s)
    k, v = _decode(s["pages_k"], s), _decode(s["pages_v"], s)
    if c["kind"] == "read":
        k = _rotate(k, s) if c["rot"] else k
        out = {"k": k.bfloat16(), "v": v.bfloat16()}
        return {**out, "means": _block_means(k)} if c["means"] else out
    q = s["q"].float().unflatten(1, (c["H"], c["g"]))
    score = torch.einsum("thgd,nhd->thgn", q, k) / math.sqrt(c["d"])
    score = score.masked_fill(torch.arange(k.shape[0], device="cuda") >= s["n_rows"], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("thgn,nhd->thgd", p / total, v)
    return {"out": o.flatten(1, 2).to(s["out"].dtype), "lse": (top + total.log()).squeeze(-1).flatten(1, 2)}


# ------------------------------------------------------------------ the package's operators

def _own(s):
    import hybrid_sparse_attention_hkv_b200 as hsa
    c = s["case"]
    if "rope" not in s and c.get("rot"):  # what a program keeps: the descriptors of its rotary positions and its pages
        layout = hsa.ROPE_HALF if c["layout"] == "half" else hsa.ROPE_INTERLEAVED
        s["rope"] = hsa.make_rope(s["inv_freq"], layout, axis_pairs=s["axis_pairs"], mscale=s["mscale"])
    if c["kind"] in ("rope", "rope_bwd"):
        call = hsa.hsa_rope if c["kind"] == "rope" else hsa.hsa_rope_bwd
        call(s["rope"], s["pos"], s["q"], s["q_out"], s["k"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if "quant" not in s:
        fmt = {"e4m3": hsa.QUANT_E4M3, "int8": hsa.QUANT_INT8, "int4": hsa.QUANT_INT4}[c["fmt"]]
        s["quant"] = hsa.make_quant(fmt, c["group"])
        size = hsa.hkv_attn_quant_workspace_size(c["T"], c["H"] * c["g"], c["H"], c["d"], c["Kp"], c["P"]) if c["kind"] == "attn" else 256
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    if c["kind"] == "write":
        hsa.hkv_quant_rows(s["quant"], s["k"], s["v"], s["table_k"], s["table_v"], c["P"], c["first"], s["ws"], rope=s.get("rope"),
                           pos=s.get("pos"))
        return _written(s)
    if c["kind"] == "read":
        hsa.hkv_gather_quant(s["quant"], s["table_k"], s["table_v"], s["sel"], c["Kp"], c["P"], c["H"], c["d"], s["kc"], s["vc"], s["ws"],
                             kbar128=s["means"], rope=s.get("rope"), pos=s.get("pos"))
        out = {"k": s["kc"], "v": s["vc"]}
        return {**out, "means": s["means"]} if c["means"] else out
    hsa.hkv_attn_quant(s["quant"], s["q"], s["table_k"], s["table_v"], s["sel"], c["Kp"], c["P"], c["H"], s["out"], s["lse"], s["ws"],
                       n_rows=s["n_rows"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits

def _turned64(x, s, conjugate=False):
    """The rotation as a product of complex numbers in 64 bits."""
    c, half = s["case"], s["case"]["rot"] // 2
    x = x.double()
    angle = s["inv_freq"][None] * s["pos"].double()[s["axis_of_pair"]].T
    turn = torch.polar(torch.full_like(angle, s["mscale"]), -angle if conjugate else angle)[:, None]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (half, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.transpose(-1, -2) if c["layout"] == "half" else z
    return torch.cat([z.flatten(-2), rest], -1)


def _stored64(x, c):
    """Codes as numbers, and scales, of 64-bit rows [T, H, d]: the nearest value that the format has, ties to even."""
    q = x.reshape(*x.shape[:-1], c["d"] // c["group"], c["group"])
    amax = q.abs().max(-1).values
    scale = torch.where(amax < TINY, torch.zeros_like(amax), amax / QMAX[c["fmt"]])
    r = torch.where(scale[..., None] > 0, q / scale[..., None], torch.zeros_like(q))
    if c["fmt"] == "e4m3":  # 3 bits behind the leading one, down to steps of 2^-9
        step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)
        r = (r / step).round() * step
    else:
        r = r.round()
    return r.reshape(x.shape), scale


def _read64(pages, s):
    c = s["case"]
    parts = []
    for p in s["sel"].tolist():
        raw, scale = pages[p], _scale_view(pages, c)[p].double()
        raw = raw[:int(_code_bytes(c))].long()
        if c["fmt"] == "int4":
            raw = torch.stack([raw % 16, raw // 16], 1).flatten()
            x = torch.where(raw > 7, raw - 16, raw).double()
        elif c["fmt"] == "int8":
            x = torch.where(raw > 127, raw - 256, raw).double()
        else:
            e, m = raw // 8 % 16, (raw % 8).double()
            x = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
            x = torch.where(raw > 127, -x, x)
        parts.append(x.reshape(c["P"], c["H"], -1, c["group"]) * scale[..., None])
    return torch.cat(parts).reshape(c["Kp"] * c["P"], c["H"], c["d"])


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] in ("rope", "rope_bwd"):
        return {n: _turned64(s[n], s, c["kind"] == "rope_bwd") for n in ("q", "k")}
    if c["kind"] == "write":
        if c["fmt"] == "int8":
            words = {"k": None, "v": None}
        out = {}
        for n, x in (("k", _turned64(s["k"], s) if c["rot"] else s["k"].double()), ("v", s["v"].double())):
            codes, scale = _stored64(x, c)
            full = torch.zeros(c["NP"] * c["P"], c["H"], c["d"], dtype=torch.float64, device="cuda")
            scales = torch.zeros(c["NP"] * c["P"], c["H"], c["d"] // c["group"], dtype=torch.float64, device="cuda")
            full[c["first"]:c["first"] + c["T"]], scales[c["first"]:c["first"] + c["T"]] = codes, scale
            out[n], out[n + "_scale"] = full.unflatten(0, (c["NP"], c["P"])), scales.unflatten(0, (c["NP"], c["P"]))
        return {**out, **words} if c["fmt"] == "int8" else out
    k, v = _read64(s["pages_k"], s), _read64(s["pages_v"], s)
    if c["kind"] == "read":
        if c["rot"]:
            k = _turned64(k, s)
        out = {"k": k, "v": v}
        if c["means"]:
            out["means"] = _block_means(k)
        return out
    k, v = k[:c["n"]], v[:c["n"]]
    q = s["q"].double().reshape(c["T"], c["H"], c["g"], c["d"])
    out, lse = [], []
    for h in range(c["H"]):
        score = q[:, h] @ k[:, h].T / math.sqrt(c["d"])
        lse.append(torch.logsumexp(score, -1))
        out.append(torch.softmax(score, -1) @ v[:, h])
    return {"out": torch.stack(out, 1).flatten(1, 2), "lse": torch.stack(lse, 1).flatten(1, 2)}
