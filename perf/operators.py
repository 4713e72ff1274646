"""Speculative decoding over a quantized KV cache: the four operators of one step, and what they cost.

A step drafts a small tree of tokens for every sequence, lets the target model look at all of them at
once and keeps the path that its probabilities accept:

  norm_rope  queries and keys of the fused projection normed per head and rotated to their positions,
             keys and values laid out as the cache's append takes them
  tree       attention of the tree's nodes over the quantized cache and over their own ancestors
  verify     the accepted path and the next token, from the probabilities and given random numbers
  append     the accepted nodes' keys and values written to the cache

``run`` computes them with elementary torch operations where ``own`` is false, and with the package's
calls where it is true.  Node 0 of a tree is its root (the last token that was sampled); ``parents[n]`` is
below n, and -1 for a root.
"""
import math

import torch

own = False

D = 128  # channels of a head
BITS = {"int2": 2, "int4": 4, "int8": 8, "fp8_e4m3": 8}


# --------------------------------------------------------------------------- #
# the cases
# --------------------------------------------------------------------------- #


def _rope(batch, n, hq, h, base, rotate_keys, pad):
    return {"op": "norm_rope", "batch": batch, "n": n, "hq": hq, "h": h, "base": float(base),
            "rotate_keys": rotate_keys, "pad": pad}


def _tree(fmt, batch, h, gh, n, lo, hi, G=0, Gv=128, R=0, S=0, paged=False):
    return {"op": "tree", "fmt": fmt, "batch": batch, "h": h, "gh": gh, "n": n, "lo": lo, "hi": hi, "G": G, "Gv": Gv,
            "R": R, "S": S, "paged": paged}


def _verify(batch, n, vocab, drafted):
    return {"op": "verify", "batch": batch, "n": n, "vocab": vocab, "drafted": drafted}


def _append(fmt, batch, h, n, lo, hi, S):
    return {"op": "append", "fmt": fmt, "batch": batch, "h": h, "n": n, "lo": lo, "hi": hi, "S": S}


def listed():
    cases = {
        # one new token per sequence, the heads of an 8B-shaped layer: a plain decode step
        "rope step": _rope(16, 1, 32, 8, 500000.0, True, 0),
        # a drafted tree per sequence on a layer that stores its keys before the rotation, padded rows
        "rope tree": _rope(7, 23, 48, 8, 10000.0, False, 64),
        # the prompts of four sequences on a 70B-shaped layer
        "rope prompts": _rope(4, 8192, 64, 8, 500000.0, True, 0),
        # the first draft after a short prompt, one sequence, an unquantized layer: the smallest call
        "tree bf16 short": _tree("bf16", 1, 2, 4, 5, 37, 37, S=1),
        # an 8B-shaped FP8 layer, 16 drafted nodes per sequence
        "tree fp8": _tree("fp8_e4m3", 16, 8, 4, 16, 8192, 8192),
        # a 70B-shaped 4-bit layer, 16 nodes: 128 query columns per kv head
        "tree int4": _tree("int4", 16, 8, 8, 16, 8192, 8192, G=128, R=128),
        # long contexts of a 2-bit layer with as many kv heads as query heads
        "tree int2 long": _tree("int2", 4, 32, 1, 32, 32768, 32768, G=32, Gv=32, R=128),
        # a ragged paged batch of an 8-bit layer with a sink token, an odd head ratio and an odd tree
        "tree int8 paged": _tree("int8", 12, 8, 6, 9, 1024, 16384, G=16, R=64, S=1, paged=True),
        # a chain of five drafted tokens for one user
        "verify chain": _verify(1, 6, 32000, True),
        # a batch of trees over a large vocabulary
        "verify trees": _verify(32, 16, 128256, True),
        # the accepted paths of the FP8 layer above, early in its sequences (the length costs nothing here)
        "append fp8": _append("fp8_e4m3", 16, 8, 16, 200, 500, 0),
        # a few sequences of an unquantized layer, odd sizes
        "append bf16": _append("bf16", 3, 5, 7, 100, 900, 1),
    }
    return [dict(c, name=name) for name, c in cases.items()]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm_rope", "tree", "tree", "verify", "append"])
    if op == "norm_rope":
        h, batch = rng.choice([1, 2, 5, 8, 32]), log(1, 32)
        return _rope(batch, log(1, max(1, 8192 // batch)), h * rng.choice([1, 2, 3, 4, 6, 8]) if h < 32 else h, h,
                     rng.choice([10000.0, 500000.0]), rng.random() < 0.7, rng.choice([0, 0, 64, 200]))
    if op == "tree":
        fmt = rng.choice(["int2", "int4", "int8", "fp8_e4m3", "bf16"])
        h, batch, n = rng.choice([1, 2, 4, 8]), log(1, 16), log(1, 64)
        gh = rng.choice([1, 2, 4, 6, 8] if n <= 32 else [1, 2, 4])
        hi = log(16, 8192)
        G = rng.choice([16, 32, 64, 128]) if fmt.startswith("int") else 0
        paged = fmt.startswith("int") and rng.random() < 0.5
        return _tree(fmt, batch, h, gh, n, rng.randint(1, hi), hi, G=G, Gv=rng.choice([32, 64, 128]) if G else 128,
                     R=rng.choice([0, 32, 64, 128]) if G else 0, S=rng.choice([0, 1, 4]), paged=paged)
    if op == "verify":
        return _verify(log(1, 32), log(1, 16), log(1000, 128256), rng.random() < 0.75)
    hi = log(64, 1000)
    return _append(rng.choice(["fp8_e4m3", "bf16"]), log(1, 16), rng.choice([1, 5, 8]), log(1, 32),
                   rng.randint(1, hi), hi, rng.choice([0, 1, 4]))


# --------------------------------------------------------------------------- #
# the cache's layout: 16-token tiles of codes in the order that a tensor-core operand is read
# --------------------------------------------------------------------------- #


def _place(bits, fp8, row, col, step):
    """Bit of the code (row, column) of `step` inside a 16 x 128 code matrix."""
    lane = 4 * (row % 8) + (col % 8) // 2
    reg, half = row // 8 + 2 * (col // 8), col % 2
    if bits == 4:
        word, at = step, 4 * reg + 16 * half
    elif bits == 2:
        word, at = step // 2, 8 * (step % 2) + 2 * reg + 16 * half
    else:
        word, at = 2 * step + reg // 2, 8 * (2 * (reg % 2) + half if fp8 else (reg % 2) + 2 * half)
    return (((word // 4) * 32 + lane) * 16 + (word % 4) * 4) * 8 + at


def _places(fmt):
    """Bit positions [16 tokens, 128 channels] of the key codes and of the value codes in a tile's part."""
    t, c = torch.arange(16, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]
    bits, fp8 = BITS[fmt], fmt.startswith("fp8")
    k = _place(bits, fp8, t + 0 * c, 2 * ((c // 4) % 4) + c % 2 + 8 * ((c % 4) // 2) + 0 * t, c // 16 + 0 * t)
    return k, _place(bits, fp8, c % 16 + 0 * t, t + 0 * c, c // 16 + 0 * t)


def _packed(codes, place, bits):
    """Codes [tiles, 16, 128] as the tiles' bytes [tiles, 2048 * bits / 8]."""
    per = 8 // bits
    order = torch.empty(16 * D, dtype=torch.int64, device="cuda")
    order[(place // bits).reshape(-1)] = torch.arange(16 * D, device="cuda")
    laid = codes.reshape(-1, 16 * D)[:, order].reshape(codes.shape[0], -1, per)
    out = laid[..., 0].clone()
    for i in range(1, per):
        out |= laid[..., i] << (bits * i)
    return out


def _codes(raw, place, bits):
    """The codes [.., 16, 128] of tiles' bytes [.., 2048 * bits / 8]."""
    return (raw[..., (place // 8).reshape(-1)] >> (place % 8).to(torch.uint8).reshape(-1)).bitwise_and_(
        (1 << bits) - 1).unflatten(-1, (16, D))


def _split(T, c):
    """Tokens of a sequence of T in the sink, in the quantized store and in the window."""
    sink = min(T, c["S"])
    n = T - sink
    if c["fmt"] == "bf16":
        return sink, 0, n
    if c["fmt"].startswith("fp8"):
        return sink, n, 0
    q = max(0, n - c["R"]) // c["G"] * c["G"]
    return sink, q, n - q


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #


def _parents(batch, n, gen):
    """Trees as a drafter grows them: a node hangs below one of the few before it."""
    back = 1 + (torch.rand(batch, n, generator=gen, device="cuda") ** 2 * 4).long()
    at = torch.arange(n, device="cuda")
    return torch.where(at > 0, (at - back).clamp_(min=0), -1).int()


def _lengths(c, gen):
    u = torch.rand(c["batch"], generator=gen, device="cuda", dtype=torch.float64)
    lo, hi = math.log(c["lo"]), math.log(c["hi"])
    return [int(x) for x in (lo + u * (hi - lo)).exp().round().tolist()]


def _affine(x, dim, levels):
    """Scale, zero point and codes of x in groups along `dim`, the way the cache's append does it."""
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s = (hi - lo) / levels
    s = torch.where(s >= 2.0 ** -126, s, torch.ones_like(s))
    z = -(lo / s)
    return s, z, (x / s + z).round_().clamp_(0, levels).to(torch.uint8)


def _records(k, v, c, place, told):
    """The store's bytes of keys and values [tokens, 128] (fp32, whole groups); `told` gets what they stand for."""
    fmt, bits, G = c["fmt"], BITS[c["fmt"]], c["G"]
    levels, ngv, n = (1 << bits) - 1, D // c["Gv"], k.shape[0]
    ks, kz, kc = _affine(k.view(n // G, G, D), 1, levels)
    vs, vz, vc = _affine(v.view(n, ngv, c["Gv"]), 2, levels)
    if told is not None:
        told += [((x.double() - z.double()) * y.double()).view(n, D) for x, y, z in ((kc, ks, kz), (vc, vs, vz))]
    tiles = [_packed(kc.reshape(-1, 16, D), place[0], bits), _packed(vc.reshape(-1, 16, D), place[1], bits)]
    tiles += [x.reshape(n // 16, 16 * ngv).view(torch.uint8) for x in (vs, vz)]
    head = torch.cat([ks, kz], 1).reshape(n // G, 2 * D).contiguous().view(torch.uint8)
    return torch.cat([head, torch.cat(tiles, 1).view(n // G, -1)], 1)


def _keys(shape, gen):
    """Keys with a few large fixed channels, as a model's are, and values."""
    k = torch.randn(*shape, D, generator=gen, device="cuda")
    v = torch.randn(*shape, D, generator=gen, device="cuda")
    big = torch.rand(D, generator=gen, device="cuda") < 0.03
    return (k * torch.where(big, 6.0, 1.0)).bfloat16(), v.bfloat16()


def _cache(c, gen, grow, told):
    """The device buffers of a layer's cache that holds `lens` tokens a sequence, with room for `grow` more.
    `told`, a list or None, gets each sequence's keys and values as the cache holds them, in 64 bits."""
    B, H, fmt, S = c["batch"], c["h"], c["fmt"], c["S"]
    lens = _lengths(c, gen)
    s = {"case": c, "lens": lens, "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    parts = [_split(T, c) for T in lens]
    most = max(max(lens), c["hi"]) + grow  # the longest sequence that the buffers are made for
    W = max(1, most) if fmt == "bf16" else 0 if fmt.startswith("fp8") else c["R"] + c["G"]
    s["W"] = W
    s["sink"] = [torch.zeros(B, H, S, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s["ring"] = [torch.zeros(B, H, W, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    if fmt != "bf16":
        s["place"] = _places(fmt)
        unit = 16 if fmt.startswith("fp8") else c["G"]
        units = [-(-p[1] // unit) for p in parts]
        ngv = D // c["Gv"]
        s["rec"] = rec = 4096 if fmt.startswith("fp8") else 8 * D + unit // 16 * (4 * D * BITS[fmt] + 128 * ngv)
        s["cap"] = cap = -(-most // unit)
        if c["paged"]:
            s["pool"] = torch.zeros(sum(units) + 3, H, rec, dtype=torch.uint8, device="cuda")
            order = torch.randperm(sum(units) + 3, generator=gen, device="cuda").int()
            s["table"] = torch.full((B, cap), -1, dtype=torch.int32, device="cuda")
            at = 0
            for b, u in enumerate(units):
                s["table"][b, :u] = order[at:at + u]
                at += u
        else:
            s["store"] = torch.zeros(B, H, cap, rec, dtype=torch.uint8, device="cuda")
    if fmt.startswith("fp8"):
        # calibrated on these very values' distribution: the largest of some hundred million normals
        s["scale"] = [torch.tensor([36.0 / 448], device="cuda"), torch.tensor([6.0 / 448], device="cuda")]
    for b, T in enumerate(lens):
        sink, q, r = parts[b]
        k, v = _keys((H, T), gen)
        for x, sk, ring in zip((k, v), s["sink"], s["ring"]):
            sk[b, :, :sink] = x[:, :sink]
            if r:
                ring[b, :, (torch.arange(q, q + r, device="cuda") % W)] = x[:, sink + q:]
        if told is not None:
            told.append([k.double(), v.double()])
        if not q:
            continue
        if fmt.startswith("fp8"):
            room = -(-q // 16) * 16
            both = []
            for i, (x, scale, place) in enumerate(zip((k, v), s["scale"], s["place"])):
                e = torch.zeros(H, room, D, dtype=torch.uint8, device="cuda")
                f = (x[:, sink:].float() / scale).clamp_(-448, 448).to(torch.float8_e4m3fn)
                e[:, :q] = f.view(torch.uint8)
                both.append(_packed(e.view(-1, 16, D), place, 8).view(H, room // 16, 2048))
                if told is not None:
                    told[-1][i][:, sink:] = f.double() * scale.double()
            rows = torch.cat(both, 2)
        else:
            held = None if told is None else []
            rows = _records(k[:, sink:sink + q].float().reshape(-1, D), v[:, sink:sink + q].float().reshape(-1, D), c,
                            s["place"], held).view(H, q // c["G"], -1)
            for i, x in enumerate(held or ()):
                told[-1][i][:, sink:sink + q] = x.view(H, q, D)
        if c["paged"]:
            s["pool"][s["table"][b, :rows.shape[1]].long()] = rows.transpose(0, 1)
        else:
            s["store"][b, :, :rows.shape[1]] = rows
    return s


def prepare(case, seed, told=None):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, c = case["op"], case
    if op == "norm_rope":
        B, n, hq, h = c["batch"], c["n"], c["hq"], c["h"]
        rows = torch.randn(B * n, (hq + 2 * h) * D + c["pad"], generator=gen, device="cuda").bfloat16()
        s = {"case": c, "rows": rows, "eps": 1e-6,
             "weights": [(1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).bfloat16() for _ in range(2)]}
        start = torch.randint(0, 100000, (B, 1), generator=gen, device="cuda")
        s["positions"] = (start + torch.arange(n, device="cuda")).int()
        s["q"] = torch.empty(B, n, hq, D, dtype=torch.bfloat16, device="cuda")
        s["k"], s["v"] = (torch.empty(B, h, n, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    elif op == "verify":
        B, n, V = c["batch"], c["n"], c["vocab"]
        logits = 3 * torch.randn(B, n, V, generator=gen, device="cuda")
        s = {"case": c, "target": logits.softmax(-1), "parents": _parents(B, n, gen),
             "u": torch.rand(B, n, generator=gen, device="cuda")}
        logits += 1.5 * torch.randn(B, n, V, generator=gen, device="cuda")
        drafted = logits.softmax(-1)
        del logits
        if c["drafted"]:  # every node drawn from the drafter's distribution at its parent
            picks = torch.multinomial(drafted.view(B * n, V), n, replacement=True, generator=gen).view(B, n, n)
            row = s["parents"].clamp(min=0).long()
            tokens = picks.gather(1, row[..., None].expand(B, n, n)).diagonal(dim1=1, dim2=2)
        else:  # the drafter's best tokens, each below its parent once
            best = drafted.topk(n, -1).indices
            same = (s["parents"][:, :, None] == s["parents"][:, None, :]).tril(-1).sum(-1)
            tokens = best[torch.arange(B, device="cuda")[:, None], s["parents"].clamp(min=0).long(), same]
        s["tokens"] = tokens.int().contiguous()
        s["draft"] = drafted if c["drafted"] else None
        s["path"] = torch.empty(B, n, dtype=torch.int32, device="cuda")
        s["accepted"], s["next"] = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    else:
        c = {"G": 0, "Gv": D, "R": 0, "paged": False, **c}
        s = _cache(c, gen, c["n"] if op == "append" else 0, told)
        B, H, n = c["batch"], c["h"], c["n"]
        s["k"], s["v"] = _keys((B, H, n), gen)
        if op == "tree":
            s["parents"] = _parents(B, n, gen)
            s["q"] = torch.randn(B, n, H * c["gh"], D, generator=gen, device="cuda").bfloat16()
            s["out"] = torch.empty_like(s["q"])
        else:  # about every third node down a path is accepted
            keep = torch.rand(B, n, generator=gen, device="cuda") < 0.4
            keep[:, 0] = True
            s["accepted"] = keep.sum(1).int()
            at = torch.where(keep, torch.arange(n, device="cuda"), n).sort(1).values
            s["path"] = torch.where(at < n, at, -1).int()
    if own:
        s["plan"] = _plan(s, op)
    return s


# --------------------------------------------------------------------------- #
# the package's calls
# --------------------------------------------------------------------------- #


def _plan(s, op):
    """What a program keeps between steps: the layer's config, its buffers' addresses, the workspace."""
    from quantized_kv_cache_decode_gb300 import kvq
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("norm_rope", "verify"):
        return kvq, status
    c = s["case"]
    fp8 = c["fmt"].startswith("fp8")
    kw = {"capacity_tokens": s["W"] if c["fmt"] == "bf16" else s["cap"] * (16 if fp8 else c["G"])}
    if c["paged"]:
        kw = {"paged": True, "block_tokens": c["G"], "num_blocks": s["pool"].shape[0], "max_blocks_per_seq": s["cap"]}
    cfg = kvq.make_config(c["fmt"], c["h"], 1 if fp8 else c["G"], c["Gv"], c["R"], c["S"], **kw)
    cache = kvq.LayerCache()
    cache.resid_k, cache.resid_v = (x.data_ptr() for x in s["ring"])
    cache.sink_k, cache.sink_v = (x.data_ptr() for x in s["sink"])
    if "store" in s:
        cache.qstore = s["store"].data_ptr()
    if "pool" in s:
        cache.block_pool, cache.block_table = s["pool"].data_ptr(), s["table"].data_ptr()
    if fp8:
        cache.k_tensor_scale, cache.v_tensor_scale = (x.data_ptr() for x in s["scale"])
    if op == "append":
        return kvq, status, cfg, cache
    size = kvq.decode_workspace_size_tree(cfg, c["batch"], c["n"], c["h"] * c["gh"])
    return kvq, status, cfg, cache, torch.zeros(size, dtype=torch.uint8, device="cuda")


def _run_own(s):
    c, p = s["case"], s["plan"]
    kvq, status = p[:2]
    if c["op"] == "norm_rope":
        kvq.qk_norm_rope(s["rows"], s["rows"].stride(0), c["batch"], c["n"], c["hq"], c["h"], *s["weights"], s["eps"],
                         s["positions"], c["base"], c["rotate_keys"], s["q"], s["k"], s["v"])
        return s["q"], s["k"], s["v"]
    if c["op"] == "verify":
        V = c["vocab"]
        kvq.verify_tree(s["target"], V, s["draft"], V, V, s["tokens"], s["parents"], s["u"], c["n"], c["batch"],
                        s["path"], s["accepted"], s["next"], status)
        return s["path"], s["accepted"], s["next"]
    cfg, cache = p[2:4]
    if c["op"] == "append":
        kvq.append_accepted(cfg, cache, s["k"], s["v"], c["n"], s["path"], s["accepted"], s["seq_lens"], c["batch"],
                            status)
        return _held(s)
    kvq.decode_attention_tree(cfg, cache, s["q"], s["k"], s["v"], s["parents"], c["n"], c["h"] * c["gh"],
                              s["seq_lens"], c["batch"], 1 / math.sqrt(D), s["out"], True, None, p[4], p[4].numel(),
                              status)
    return s["out"]


def _held(s):
    """The cache as it stands: an FP8 store as its values (in units of the layer's scales)."""
    return [x.view(torch.float8_e4m3fn) for x in [s.get("store")] if x is not None] + s["sink"] + s["ring"]


# --------------------------------------------------------------------------- #
# the plain forms
# --------------------------------------------------------------------------- #


def _turned(x, positions, base):
    """Rows [.., tokens, heads, 128] rotated: channel i and i + 64 by position * base^(-i / 64)."""
    i = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    angle = positions.double()[..., None, None] * base ** (-i / (D // 2))
    cos, sin = angle.cos().to(x.dtype), angle.sin().to(x.dtype)
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_norm_rope(s):
    c = s["case"]
    B, n, hq, h = c["batch"], c["n"], c["hq"], c["h"]
    x = s["rows"][:, :(hq + 2 * h) * D].view(B, n, hq + 2 * h, D)

    def normed(x, w):
        x = x.float()
        return x * (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * w.float()

    q, k = normed(x[:, :, :hq], s["weights"][0]), normed(x[:, :, hq:hq + h], s["weights"][1])
    q = _turned(q, s["positions"], c["base"])
    k = _turned(k, s["positions"], c["base"]) if c["rotate_keys"] else k
    return (q.bfloat16(), k.bfloat16().transpose(1, 2).contiguous(),
            x[:, :, hq + h:].transpose(1, 2).contiguous())


def _values(s, b):
    """Keys and values [heads, tokens, 128] in fp32 that sequence b's cache stands for."""
    dtype = torch.float32
    c, T = s["case"], s["lens"][b]
    sink, q, r = _split(T, c)
    parts = [[x[b, :, :sink].to(dtype)] for x in s["sink"]]
    if q:
        fp8 = c["fmt"].startswith("fp8")
        unit = 16 if fp8 else c["G"]
        units = -(-q // unit)
        rows = s["pool"][s["table"][b, :units].long()].transpose(0, 1) if c["paged"] else s["store"][b, :, :units]
        bits, ngv = BITS[c["fmt"]], D // c["Gv"]
        part = 16 * D * bits // 8
        head = 0 if fp8 else 8 * D
        tiles = rows[..., head:].unflatten(-1, (unit // 16, -1))
        kc = _codes(tiles[..., :part], s["place"][0], bits)  # [heads, units, tiles, 16, 128]
        vc = _codes(tiles[..., part:2 * part], s["place"][1], bits)
        if fp8:
            k, v = (x.contiguous().view(torch.float8_e4m3fn).to(dtype) * scale.to(dtype)
                    for x, scale in zip((kc, vc), s["scale"]))
        else:
            ks, kz = rows[..., :head].contiguous().view(torch.float32).to(dtype).unflatten(-1, (2, 1, 1, D)).unbind(2)
            vs, vz = tiles[..., 2 * part:].contiguous().view(torch.float32).to(dtype).unflatten(
                -1, (2, 16, ngv, 1)).unbind(3)
            k = (kc.to(dtype) - kz) * ks
            v = ((vc.to(dtype).unflatten(-1, (ngv, -1)) - vz) * vs).flatten(-2)
        for at, x in zip(parts, (k, v)):
            at.append(x.reshape(c["h"], units * unit, D)[:, :q])
    if r:
        slots = torch.arange(q, q + r, device="cuda") % s["W"]
        for at, x in zip(parts, s["ring"]):
            at.append(x[b][:, slots].to(dtype))
    return [torch.cat(x, 1) for x in parts]


def _ancestors(parents):
    """[batch, n, n]: whether column m is node n itself or above it."""
    n = parents.shape[1]
    at = torch.arange(n, device=parents.device)
    up = (parents[:, :, None] == at).float()
    reach = torch.eye(n, device=parents.device) + up
    for _ in range(max(1, (n - 1).bit_length())):  # paths of twice the length each time
        reach = (reach @ reach > 0).float()
    return reach > 0


def _plain_tree(s):
    c = s["case"]
    seen = _ancestors(s["parents"])
    out = torch.empty_like(s["q"])
    for b, T in enumerate(s["lens"]):
        k, v = _values(s, b)
        k, v = torch.cat([k, s["k"][b].float()], 1), torch.cat([v, s["v"][b].float()], 1)
        q = s["q"][b].float().unflatten(1, (c["h"], c["gh"])).permute(1, 2, 0, 3)  # [heads, group, nodes, 128]
        x = q.flatten(1, 2) @ k.transpose(1, 2) / math.sqrt(D)
        x = x.unflatten(1, (c["gh"], c["n"]))
        x[..., T:].masked_fill_(~seen[b], -math.inf)
        x = (x - x.amax(-1, keepdim=True)).exp_()
        y = (x / x.sum(-1, keepdim=True)).flatten(1, 2) @ v
        out[b] = y.unflatten(1, (c["gh"], c["n"])).permute(2, 0, 1, 3).flatten(1, 2).bfloat16()
    return out


def _plain_verify(s):
    """In 64 bits: a sum over the vocabulary is compared with a random number."""
    c, B, n = s["case"], s["case"]["batch"], s["case"]["n"]
    rows = torch.arange(B, device="cuda")
    at = torch.zeros(B, dtype=torch.int64, device="cuda")  # the last accepted node
    w, total = s["target"][:, 0].double(), torch.ones(B, dtype=torch.float64, device="cuda")
    u = s["u"].double()
    path = torch.full((B, n), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    count = torch.ones(B, dtype=torch.int64, device="cuda")
    for i in range(1, n):
        token = s["tokens"][:, i].long()
        tried = s["parents"][:, i] == at
        if s["draft"] is None:
            q = torch.zeros_like(w).scatter_(1, token[:, None], 1.0)
        else:
            q = s["draft"][rows, at].double()
        q = q * total[:, None]
        kept = tried & (u[:, i] * q[rows, token] < w[rows, token])
        left = (w - q).clamp_(min=0)
        lost = tried & ~kept
        w = torch.where(lost[:, None], left, w)
        total = torch.where(lost, left.sum(-1), total)
        at = torch.where(kept, i, at)
        w = torch.where(kept[:, None], s["target"][:, i].double(), w)
        total = torch.where(kept, 1.0, total)
        path.scatter_(1, count.clamp(max=n - 1)[:, None], torch.where(kept, i, path.gather(
            1, count.clamp(max=n - 1)[:, None])[:, 0])[:, None])
        count += kept
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, s["target"][rows, at].double())
    sums = w.cumsum(-1)
    chosen = (sums <= u[:, :1] * sums[:, -1:]).sum(-1)
    last = c["vocab"] - 1 - (w > 0).flip(-1).int().argmax(-1)
    return path.int(), count.int(), torch.minimum(chosen, last).int()


def _plain_append(s):
    c, S = s["case"], s["case"]["S"]
    B, H, n = c["batch"], c["h"], c["n"]
    b, j = (torch.arange(n, device="cuda") < s["accepted"][:, None]).nonzero(as_tuple=True)
    node, t = s["path"][b, j].long(), s["seq_lens"][b].long() + j
    first = t < S
    for x, sink, ring in zip((s["k"], s["v"]), s["sink"], s["ring"]):
        rows = x[b, :, node]
        sink[b[first], :, t[first]] = rows[first]
        if c["fmt"] == "bf16":
            ring[b[~first], :, t[~first] - S] = rows[~first]
    if c["fmt"] == "bf16":
        return _held(s)
    b, node, t = b[~first], node[~first], t[~first] - S
    for part, (x, scale, place) in enumerate(zip((s["k"], s["v"]), s["scale"], s["place"])):
        e = (x[b, :, node].float() / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["store"][b[:, None, None], torch.arange(H, device="cuda")[:, None], (t // 16)[:, None, None],
                   part * 2048 + place[t % 16][:, None] // 8] = e
    return _held(s)


def run(state):
    if own:
        return _run_own(state)
    return {"norm_rope": _plain_norm_rope, "tree": _plain_tree, "verify": _plain_verify,
            "append": _plain_append}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- #
# the definition in 64 bits, and the work
# --------------------------------------------------------------------------- #


def _exact_norm_rope(s):
    c = s["case"]
    B, n, hq, h = c["batch"], c["n"], c["hq"], c["h"]
    i = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[..., None] * torch.exp(-i * (math.log(c["base"]) / 64)))

    def heads(lo, hi, w, rotate):
        out = torch.empty(B, n, hi - lo, D, dtype=torch.float64, device="cuda")
        for a in range(lo, hi):
            x = s["rows"][:, a * D:(a + 1) * D].double().view(B, n, D)
            if w is not None:
                x = w.double() * x / torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / D + s["eps"])
            if rotate:
                y = torch.complex(x[..., :64], x[..., 64:]) * turn
                x = torch.cat([y.real, y.imag], -1)
            out[:, :, a - lo] = x
        return out

    return (heads(0, hq, s["weights"][0], True),
            heads(hq, hq + h, s["weights"][1], c["rotate_keys"]).transpose(1, 2).contiguous(),
            heads(hq + h, hq + 2 * h, None, False).transpose(1, 2).contiguous())


def _exact_tree(s, told):
    c = s["case"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, T in enumerate(s["lens"]):
        above = []
        for node, up in enumerate(s["parents"][b].tolist()):
            above.append((above[up] if up >= 0 else []) + [node])
        k, v = told[b]
        for h in range(c["h"]):
            q = s["q"][b, :, h * c["gh"]:(h + 1) * c["gh"]].double()  # [nodes, group, 128]
            past = torch.einsum("ngd,td->ngt", q, k[h])
            for node, seen in enumerate(above):
                new = torch.einsum("gd,td->gt", q[node], s["k"][b, h, seen].double())
                p = torch.softmax(torch.cat([past[node], new], -1) * D ** -0.5, -1)
                out[b, node, h * c["gh"]:(h + 1) * c["gh"]] = p[:, :T] @ v[h] + p[:, T:] @ s["v"][b, h, seen].double()
    return out


def exact(case, seed):
    if case["op"] == "verify":  # nodes and tokens, no computed numbers
        return None
    told = []
    s = prepare(case, seed, told if case["op"] == "tree" else None)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(s)
    if case["op"] == "tree":
        return _exact_tree(s, told)
    lens, counts, path = s["lens"], s["accepted"].tolist(), s["path"].tolist()
    held = [None if x is None else x.double() for x in _held(s)]
    sinks, rings = held[-4:-2], held[-2:]
    for b, T in enumerate(lens):
        for j in range(counts[b]):
            t, node = T + j, path[b][j]
            for part, x in enumerate((s["k"], s["v"])):
                if t < case["S"]:
                    sinks[part][b, :, t] = x[b, :, node].double()
                elif case["fmt"] == "bf16":
                    rings[part][b, :, t - case["S"]] = x[b, :, node].double()
                else:
                    at = t - case["S"]
                    y = x[b, :, node].double() / s["scale"][part].double()
                    held[0][b, :, at // 16, part * 2048 + s["place"][part][at % 16] // 8] = y
    return held


def work(case):
    c, op = case, case["op"]
    if op == "norm_rope":
        rows = c["batch"] * c["n"]
        return {"bytes": rows * (4 * D * (c["hq"] + 2 * c["h"]) + 4), "flops": rows * 10 * D * (c["hq"] + c["h"])}
    if op == "verify":  # the rows of the last accepted node: the next token is drawn from them
        return {"bytes": c["batch"] * c["vocab"] * (8 if c["drafted"] else 4), "flops": 3 * c["batch"] * c["vocab"]}
    if op == "append":  # about every third node's keys and values
        kept = c["batch"] * c["h"] * (1 + 0.4 * (c["n"] - 1))
        return {"bytes": kept * D * 2 * (3 if c["fmt"].startswith("fp8") else 4), "flops": kept * D * 4}
    mean = c["lo"] if c["lo"] == c["hi"] else (c["hi"] - c["lo"]) / math.log(c["hi"] / c["lo"])
    if c["fmt"] == "bf16":
        per = 4 * D
    elif c["fmt"].startswith("fp8"):
        per = 2 * D
    else:
        per = 2 * D * BITS[c["fmt"]] / 8 + 8 * D / c["G"] + 8 * D / c["Gv"]
    pairs = c["batch"] * c["h"]
    return {"bytes": pairs * (mean * per + c["n"] * D * (4 + 4 * c["gh"])),
            "flops": pairs * 4.0 * D * c["gh"] * c["n"] * (mean + c["n"] / 2)}
