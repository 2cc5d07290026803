"""Serving operators around the quantized paged KV cache: sizes, inputs, plain forms.

Five operators of one speculative serving step over the cache of include/kvq.h:

  rope        rotary position embedding of query and key rows (half and interleaved
              layouts, part of the head, frequencies scaled for long contexts);
  rope_write  the same rotation fused with quantize-on-write of K and V into the pages;
  gather      cached rows read back by slot as K and V rows of the activation type;
  tree        attention of a tree of drafted tokens per sequence, over the cached prefix
              and, through a bit mask, the draft's own ancestors;
  commit      the accepted path's cache rows moved to the positions they are accepted at.

A case is a dict of sizes; `prepare` makes its inputs from a seed, `run` is one pass (the
plain form in elementary torch operations, or the library's call where `own` is true),
`exact` the result from the definition in 64 bits, `work` the bytes and operations that
one pass cannot do without.
"""

import math

import torch

own = False

_ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_GROUP = 64          # INT4: tokens of a key group (one block), channels of a value group


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's queries and keys of 24 sequences (64 / 8 heads), before an
        # append to a low-bit cache: the smallest call, latency counts
        _rope("rope-decode", 24, 64, 8, "half", 128, "wavelength"),
        # an odd-sized prefill of fused QKV rows, half of each head rotated, interleaved
        # pairs, context stretched by a ramp over the frequencies
        _rope("rope-prefill", 16411, 32, 8, "interleaved", 64, "yarn"),
        # one decode step into an FP8 cache with static per-head scales (64 sequences)
        _rope_write("write-decode-fp8", 64, 32, 8, "fp8", "half", 128, "none"),
        # four 8192-token prefill chunks into an INT8 cache with a scale per token and head,
        # and the chunk's rows read back for a layer that wants them whole
        _rope_write("write-prefill-int8", 32768, 64, 8, "int8", "half", 128, "linear"),
        # a cached prefix of 2048 tokens read back (32 kv heads, INT8), as for a transfer
        _gather("gather-int8", 2048, 32, "int8"),
        # a whole 32640-token INT4 prefix (groups of 64) read back
        _gather("gather-int4", 32640, 8, "int4"),
        # one user, a tree of 8 drafted tokens over a short INT8 context: latency counts
        _tree("tree-small", 1, 32, 8, "int8", 1032, 1032, 8, 8),
        # 64 users with contexts of 1 to 8 thousand tokens (FP8), ragged trees
        _tree("tree-ragged-fp8", 64, 32, 8, "fp8", 1024, 8192, 1, 32),
        # 24 users at 16384 tokens (INT8), trees of 16: one full tile of query rows each
        _tree("tree-long-int8", 24, 64, 8, "int8", 16384, 16384, 16, 16),
        # wide trees of 64 over an unquantized cache: bound by the matrix products
        _tree("tree-wide-bf16", 8, 64, 8, "bf16", 16384, 16384, 64, 64),
        # the accepted path of 24 trees of 16 (INT8)
        _commit("commit-int8", 24, 8, "int8", 16, 6),
        # the accepted paths of 256 trees of 64 over a 32-head bf16 cache
        _commit("commit-bf16", 256, 32, "bf16", 64, 16),
    ]


def _rope(name, tokens, hq, hkv, layout, rot, scaling):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": hq, "kv_heads": hkv, "dim": 128,
            "layout": layout, "rot": rot, "scaling": scaling, "act": "bf16"}


def _rope_write(name, tokens, hq, hkv, cache, layout, rot, scaling):
    return {"name": name, "op": "rope_write", "tokens": tokens, "q_heads": hq, "kv_heads": hkv, "dim": 128,
            "cache": cache, "layout": layout, "rot": rot, "scaling": scaling, "act": "bf16"}


def _gather(name, tokens, hkv, cache):
    return {"name": name, "op": "gather", "tokens": tokens, "kv_heads": hkv, "dim": 128, "cache": cache,
            "act": "bf16"}


def _tree(name, batch, hq, hkv, cache, n_low, n_high, l_low, l_high):
    return {"name": name, "op": "tree", "batch": batch, "q_heads": hq, "kv_heads": hkv, "dim": 128,
            "cache": cache, "n_low": n_low, "n_high": n_high, "l_low": l_low, "l_high": l_high, "act": "bf16"}


def _commit(name, batch, hkv, cache, tree, accept):
    return {"name": name, "op": "commit", "batch": batch, "kv_heads": hkv, "dim": 128, "cache": cache,
            "tree": tree, "accept": accept, "act": "bf16"}


def draw(rng):
    def size(low, high):                       # spread over the logarithm
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    op = rng.choice(["rope", "rope_write", "gather", "tree", "tree", "commit"])
    hkv = rng.choice([2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    layout = rng.choice(["half", "interleaved"])
    rot = rng.choice([32, 64, 96, 128])
    scaling = rng.choice(["none", "linear", "ntk", "wavelength", "yarn"])
    if op == "rope":
        c = _rope("", size(1, 16384), hq, hkv, layout, rot, scaling)
    elif op == "rope_write":
        c = _rope_write("", size(1, 16384), hq, hkv, rng.choice(["int8", "fp8", "bf16"]), layout, rot, scaling)
    elif op == "gather":
        c = _gather("", size(1, 32640), hkv, rng.choice(["int8", "fp8", "bf16", "int4"]))
    elif op == "tree":
        batch = size(1, 64)
        high = size(128, min(16384, 393216 // batch))
        most = min(64, high, (8 * 16384 * 64 * 64) // (batch * high * hq))
        l_high = size(1, max(1, most))
        c = _tree("", batch, hq, hkv, rng.choice(["int8", "fp8", "bf16"]), max(l_high, high // rng.choice([1, 2, 8])),
                  high, rng.choice([1, l_high]), l_high)
    else:
        tree = size(4, 64)
        c = _commit("", size(1, 256), hkv, rng.choice(["int8", "fp8", "bf16"]), tree, rng.randint(1, max(1, tree // 4)))
    c["act"] = rng.choice(["bf16", "fp16"]) if c.get("cache") != "bf16" else "bf16"
    del c["name"]
    return c


# ------------------------------------------------------------------------ cache layout
# One record per (block, kv head): K codes [bs][row], V codes [bs][row], then scales (float32
# K [bs] and V [bs] for int8; float16 parameters for int4), padded to 128 bytes.
def _layout(c):
    D, kind = c["dim"], c["cache"]
    bs = 64 if kind == "int4" else 16
    row = {"bf16": 2 * D, "int8": D, "fp8": D, "int4": D // 2}[kind]
    extra = {"bf16": 0, "int8": 8 * bs, "fp8": 0, "int4": 4 * D + bs * (D // _GROUP) * 4}[kind]
    rec = (2 * bs * row + extra + 127) // 128 * 128
    return bs, row, rec


class _Views:
    """Typed views into a pool of records [blocks][heads][record bytes]."""

    def __init__(self, pool, c, blocks):
        bs, row, rec = _layout(c)
        H, D, kind = c["kv_heads"], c["dim"], c["cache"]

        def at(dtype, offset, shape, strides):
            t = pool.view(dtype)
            z = t.element_size()
            return t.as_strided((blocks, H) + shape, (H * rec // z, rec // z) + strides, offset // z)

        code = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}[kind]
        n = row // torch.empty((), dtype=code).element_size()
        self.k = at(code, 0, (bs, n), (n, 1))
        self.v = at(code, bs * row, (bs, n), (n, 1))
        if kind == "int8":
            self.ks = at(torch.float32, 2 * bs * row, (bs,), (1,))
            self.vs = at(torch.float32, 2 * bs * row + 4 * bs, (bs,), (1,))
        if kind == "int4":
            g = D // _GROUP
            self.kz = at(torch.float16, 2 * bs * row, (2, D), (D, 1))             # scale, zero per channel
            self.vz = at(torch.float16, 2 * bs * row + 4 * D, (bs, g, 2), (2 * g, 2, 1))


def _int4_groups(x, dim):
    """INT4 codes of x over groups along `dim` (kept), their float16 scale and zero point."""
    lo, hi = x.amin(dim, keepdim=True).clamp(max=0), x.amax(dim, keepdim=True).clamp(min=0)
    s = ((hi - lo) / 15).half()
    w = s.float()
    z = torch.where(w > 0, torch.round(-lo / w.clamp(min=1e-30)), torch.zeros_like(w)).clamp(0, 15)
    code = torch.where(w > 0, torch.round(x / w.clamp(min=1e-30)) + z, torch.zeros_like(x)).clamp(0, 15)
    return code.to(torch.uint8), s, z.half()


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _fill(pool, c, blocks, gen):
    """Fill every block with rows of unit normal values (keys with four channels ten times
    as large), quantized as the cache's writer does; static FP8 scales come back."""
    bs, row, rec = _layout(c)
    H, D, kind, dev = c["kv_heads"], c["dim"], c["cache"], pool.device
    w = _Views(pool, c, blocks)
    wide = torch.ones(H, 1, D, device=dev)
    wide[:, :, torch.randperm(D, generator=gen, device=dev)[:4]] = 10.0
    scale = torch.tensor([10 * 4.5 / 448, 4.5 / 448], device=dev)[:, None].repeat(1, H).contiguous()
    step = max(1, (1 << 26) // (H * bs * D))
    for b in range(0, blocks, step):
        m = min(step, blocks - b)
        for i, codes in enumerate((w.k, w.v)):
            x = torch.randn(m, H, bs, D, generator=gen, device=dev)
            x = (x * wide if i == 0 else x).to(_ACT[c["act"]]).float()
            if kind == "bf16":
                codes[b:b + m] = x.to(torch.bfloat16)
            elif kind == "fp8":
                codes[b:b + m] = (x / scale[i][:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            elif kind == "int8":
                s = x.abs().amax(-1) / 127
                codes[b:b + m] = torch.round(x / s[..., None]).clamp(-128, 127).to(torch.int8)
                (w.ks if i == 0 else w.vs)[b:b + m] = s
            elif i == 0:
                code, s, z = _int4_groups(x, 2)
                codes[b:b + m] = _pack(code)
                w.kz[b:b + m, :, 0], w.kz[b:b + m, :, 1] = s[:, :, 0], z[:, :, 0]
            else:
                code, s, z = _int4_groups(x.view(m, H, bs, D // _GROUP, _GROUP), 4)
                codes[b:b + m] = _pack(code.view(m, H, bs, D))
                w.vz[b:b + m, ..., 0], w.vz[b:b + m, ..., 1] = s[..., 0], z[..., 0]
    return scale


def _pool(c, blocks, dev):
    return torch.zeros(blocks * c["kv_heads"] * _layout(c)[2], dtype=torch.uint8, device=dev)


# --------------------------------------------------------------------------- inputs
def _scaling(c):
    """What the frequencies are stretched by: contexts of 8192 tokens to eight times that."""
    none = {"kind": c["scaling"], "theta": 500000.0, "factor": 8.0, "original": 8192, "low": 1.0, "high": 1.0}
    return {**none, **{"wavelength": {"low": 1.0, "high": 4.0}, "yarn": {"low": 1.0, "high": 32.0}}.get(c["scaling"], {})}


def _frequencies(c):
    """Radians per position of every pair, float64, and what cosine and sine are multiplied by."""
    s, rot = _scaling(c), c["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    theta, by = s["theta"], 1.0
    if s["kind"] == "ntk":
        theta = theta * s["factor"] ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if s["kind"] == "linear":
        f = f / s["factor"]
    elif s["kind"] == "wavelength":
        turns = s["original"] * f / (2 * math.pi)          # turns within the original context
        t = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        f = (1 - t) * f / s["factor"] + t * f
    elif s["kind"] == "yarn":
        def dim(turns):
            return rot * math.log(s["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))

        a, b = max(math.floor(dim(s["high"])), 0), min(math.ceil(dim(s["low"])), rot - 1)
        t = 1 - ((i - a) / max(b - a, 0.001)).clamp(0, 1)
        f = (1 - t) * f / s["factor"] + t * f
        by = 0.1 * math.log(s["factor"]) + 1
    return f, by


def _random_tree(size, gen):
    """Ancestor rows of a random tree of drafted tokens: bit j of row i is set where token i
    sees token j (itself and its ancestors).  Token 0 is the root."""
    parent = [-1] + [i - 1 if float(torch.rand((), generator=gen)) < 0.4 else
                     int(torch.randint(0, i, (), generator=gen)) for i in range(1, size)]
    rows = torch.zeros(size, size, dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            rows[i] = rows[p]
        rows[i, i] = True
    return rows


def _spread(low, high, count, gen):
    """`count` sizes spread evenly over [low, high], in random order: their sum is the case's."""
    return torch.linspace(low, high, count).round().long()[torch.randperm(count, generator=gen)]


def _words(rows, words):
    """Boolean rows packed into int32 words, bit j % 32 of word j // 32."""
    bits = torch.zeros(rows.shape[0], 32 * words, dtype=torch.int64)
    bits[:, :rows.shape[1]] = rows.long()
    packed = (bits.view(-1, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": c}
    D, act = c["dim"], _ACT[c["act"]]
    if c["op"] in ("rope", "rope_write"):
        # fused projection rows: the heads of q, then those of k, then those of v
        T, hq, hkv = c["tokens"], c["q_heads"], c["kv_heads"]
        qkv = torch.randn(T, (hq + 2 * hkv) * D, generator=gen, device=dev).to(act)
        s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
        s["k"] = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        s["v"] = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        s["positions"] = torch.randint(0, 65536, (T,), generator=gen, device=dev, dtype=torch.int32)
        f, s["by"] = _frequencies(c)
        s["freqs"] = f.to(dev)
    if c["op"] == "rope_write":
        blocks = c["tokens"] // 16 + 2
        s["pool"] = _pool(c, blocks, dev)
        s["blocks"] = blocks
        s["slots"] = torch.randperm(16 * blocks, generator=gen, device=dev)[:c["tokens"]].to(torch.int32)
        s["scale"] = torch.full((2, c["kv_heads"]), 4.5 / 448, device=dev)
    if c["op"] == "gather":
        bs = _layout(c)[0]
        blocks = c["tokens"] // bs + 2
        s["pool"], s["blocks"] = _pool(c, blocks, dev), blocks
        s["scale"] = _fill(s["pool"], c, blocks, gen)
        table = torch.randperm(blocks, generator=gen, device=dev)
        t = torch.arange(c["tokens"], device=dev)
        s["slots"] = (table[t // bs] * bs + t % bs).to(torch.int32)
    if c["op"] in ("tree", "commit"):
        B = c["batch"]
        if c["op"] == "tree":
            lens, size = _spread(c["n_low"], c["n_high"], B, host), _spread(c["l_low"], c["l_high"], B, host)
            most, top = c["l_high"], c["n_high"]
        else:
            size = torch.full((B,), c["tree"])
            lens = size + _spread(1, 48, B, host)
            most, top = c["tree"], c["tree"] + 48
        per = (top + 15) // 16
        used = ((lens + 15) // 16).sum().item()
        blocks = used + 3
        table = torch.randperm(blocks, generator=host)[:used].to(torch.int32)
        tables = torch.zeros(B, per, dtype=torch.int32)
        tables[torch.arange(per) < ((lens + 15) // 16)[:, None]] = table
        s["pool"], s["blocks"] = _pool(c, blocks, dev), blocks
        s["scale"] = _fill(s["pool"], c, blocks, gen)
        s["tables"], s["lens"] = tables.to(dev), lens.to(torch.int32).to(dev)
        s["start"] = torch.cat([torch.zeros(1, dtype=torch.long), size.cumsum(0)]).to(torch.int32).to(dev)
        s["most"], s["top"] = most, top
    if c["op"] == "tree":
        words = (most + 31) // 32
        trees = [_random_tree(most, host) for _ in range(4)]          # a sequence takes one of four shapes
        packed = [_words(t, words) for t in trees]
        s["mask"] = torch.cat([packed[b % 4][:int(size[b])] for b in range(B)]).to(dev)
        s["q"] = torch.randn(int(size.sum()), c["q_heads"], D, generator=gen, device=dev).to(act)
    if c["op"] == "commit":
        # the root is always accepted and stays; later tokens of the path lie beyond the places
        # that the path moves to, so that a second pass on the same pool changes nothing
        a = torch.randint(1, c["accept"] + 1, (B,), generator=host)
        path = torch.zeros(B, c["accept"], dtype=torch.long)
        room = c["tree"] - c["accept"]
        for b in range(B):
            pick = torch.randperm(room, generator=host)[:c["accept"] - 1].sort().values + c["accept"]
            path[b, 1:] = pick
        s["path"], s["accepted"] = path.to(torch.int32).to(dev), a.to(torch.int32).to(dev)
    return s


# ------------------------------------------------------------------------- plain forms
def _rotated(s, x):
    """x [T][H][D] rotated, float32: pair p of a head turns by position * frequency p."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = (angle.cos() * s["by"]).float()[:, None], (angle.sin() * s["by"]).float()[:, None]
    x = x.float()
    turn, rest = x[..., :rot], x[..., rot:]
    if c["layout"] == "half":
        a, b = turn[..., :half], turn[..., half:]
        turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turn, rest], -1)


def _read(s, blk, head, off):
    """Values of K and V at (block, head, offset) index tensors, float32."""
    c, w = s["case"], _Views(s["pool"], s["case"], s["blocks"])
    kind = c["cache"]
    if kind == "bf16":
        return w.k[blk, head, off].float(), w.v[blk, head, off].float()
    if kind == "int8":
        return (w.k[blk, head, off].float() * w.ks[blk, head, off][..., None],
                w.v[blk, head, off].float() * w.vs[blk, head, off][..., None])
    if kind == "fp8":
        k = w.k.view(torch.uint8)[blk, head, off].view(torch.float8_e4m3fn).float()
        v = w.v.view(torch.uint8)[blk, head, off].view(torch.float8_e4m3fn).float()
        return k * s["scale"][0][head][..., None], v * s["scale"][1][head][..., None]

    def unpack(codes):
        return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()

    kz, vz = w.kz[blk, head].float(), w.vz[blk, head, off].float().repeat_interleave(_GROUP, -2)
    return ((unpack(w.k[blk, head, off]) - kz[..., 1, :]) * kz[..., 0, :],
            (unpack(w.v[blk, head, off]) - vz[..., 1]) * vz[..., 0])


def _slot_index(s):
    bs = _layout(s["case"])[0]
    slots = s["slots"].long()
    return (slots // bs)[:, None], torch.arange(s["case"]["kv_heads"], device=slots.device)[None], (slots % bs)[:, None]


def _plain_rope(s):
    return [_rotated(s, s["q"]).to(s["q"].dtype), _rotated(s, s["k"]).to(s["k"].dtype)]


def _plain_rope_write(s):
    c, at = s["case"], _slot_index(s)
    w = _Views(s["pool"], c, s["blocks"])
    q, k, v = _rotated(s, s["q"]).to(s["q"].dtype), _rotated(s, s["k"]), s["v"].float()
    if c["cache"] == "bf16":
        w.k[at], w.v[at] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        return [q, s["pool"].view(torch.bfloat16)]
    if c["cache"] == "fp8":
        for codes, x, scale in ((w.k, k, s["scale"][0]), (w.v, v, s["scale"][1])):
            code = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            codes.view(torch.uint8)[at] = code.view(torch.uint8)
        return [q, s["pool"].view(torch.float8_e4m3fn)]
    for codes, scales, x in ((w.k, w.ks, k), (w.v, w.vs, v)):
        scale = x.abs().amax(-1) / 127
        codes[at] = torch.round(x / scale[..., None]).clamp(-128, 127).to(torch.int8)
        scales[at] = scale
    k, v = _read(s, *at)
    return [q, k.to(s["k"].dtype), v.to(s["v"].dtype)]


def _plain_gather(s):
    k, v = _read(s, *_slot_index(s))
    return [k.to(_ACT[s["case"]["act"]]), v.to(_ACT[s["case"]["act"]])]


def _visible(s, row, size):
    """[B][most][top] which positions each query of each sequence sees."""
    lens, most, top = s["lens"].long(), s["most"], s["top"]
    at = torch.arange(top, device=lens.device)
    first = (lens - size)[:, None]
    j = (at[None] - first).clamp(0, most - 1)
    word = s["mask"].long()[row.clamp(max=s["mask"].shape[0] - 1)]
    bit = (word[..., None] >> torch.arange(32, device=lens.device)) & 1
    tree = torch.gather(bit.flatten(-2), 2, j[:, None].expand(-1, most, -1)) > 0
    return (at[None, None] < lens[:, None, None]) & ((at[None] < first)[:, None] | tree)


def _plain_tree(s):
    c = s["case"]
    B, H, D, most, top = c["batch"], c["kv_heads"], c["dim"], s["most"], s["top"]
    g, dev = c["q_heads"] // H, s["q"].device
    at = torch.arange(top, device=dev)
    blk = s["tables"].long()[:, at // 16]
    head = torch.arange(H, device=dev)[None, :, None]
    k, v = _read(s, blk[:, None], head, (at % 16)[None, None])                 # [B][H][top][D]
    start = s["start"].long()
    size = start[1:] - start[:-1]
    row = start[:-1, None] + torch.arange(most, device=dev)                      # [B][most]
    have = torch.arange(most, device=dev) < size[:, None]
    q = s["q"].float()[row.clamp(max=s["q"].shape[0] - 1)].view(B, most, H, g, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, H, most * g, D)
    see = _visible(s, row, size)[:, None, :, None].expand(-1, -1, -1, g, -1).reshape(B, 1, most * g, top)
    z = torch.matmul(q, k.transpose(-1, -2)).div_(math.sqrt(D)).masked_fill_(~see, -math.inf)
    z = z.sub_(z.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    o = torch.matmul(z, v) / z.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(B, H, most, g, D).permute(0, 2, 1, 3, 4).reshape(B, most, H * g, D)
    return [o[have].to(s["q"].dtype)]


def _plain_commit(s):
    c = s["case"]
    w = _Views(s["pool"], c, s["blocks"])
    start, lens = s["start"].long(), s["lens"].long()
    first = lens - (start[1:] - start[:-1])
    j = torch.arange(c["accept"], device=lens.device)[None]
    b, j = torch.nonzero(j < s["accepted"][:, None], as_tuple=True)
    src, dst = first[b] + s["path"].long()[b, j], first[b] + j
    head = torch.arange(c["kv_heads"], device=lens.device)[None]
    src_at = (s["tables"].long()[b, src // 16][:, None], head, (src % 16)[:, None])
    dst_at = (s["tables"].long()[b, dst // 16][:, None], head, (dst % 16)[:, None])
    parts = [w.k, w.v] + ([w.ks, w.vs] if c["cache"] == "int8" else [])
    parts = [p.view(torch.uint8) if p.dtype == torch.float8_e4m3fn else p for p in parts]
    rows = [p[src_at] for p in parts]
    for p, r in zip(parts, rows):
        p[dst_at] = r
    return [_whole_pool(s), (first + s["accepted"].long()).to(torch.int32)]


def _whole_pool(s):
    return s["pool"].view(torch.bfloat16) if s["case"]["cache"] == "bf16" else s["pool"]


# ------------------------------------------------------------------- the library's calls
def _handles(s):
    """What a serving program keeps beside the pool: the cache and rope handles, the workspace."""
    if "cache" in s or "rope" in s:
        return
    from quantized_paged_kv_02_b200 import kvq
    c = s["case"]
    if c["op"] in ("rope", "rope_write"):
        p = _scaling(c)
        s["rope"] = kvq.Rope(c["dim"], c["rot"], theta=p["theta"], layout=c["layout"], scaling=p["kind"],
                             factor=p["factor"], original_context=p["original"], low=p["low"], high=p["high"])
    if c["op"] == "rope":
        return
    mode = {"bf16": "none", "int8": "per_token_head", "fp8": "per_head", "int4": "kivi"}[c["cache"]]
    s["cache"] = kvq.PagedKVCache(c["cache"], c["act"], mode, s["blocks"], _layout(c)[0], c["kv_heads"], c["dim"],
                                  pages=s["pool"], max_seqs=1 if c["cache"] == "int4" else 0,
                                  static_k_scale=s["scale"][0], static_v_scale=s["scale"][1])
    if c["op"] == "tree":
        n = s["cache"].tree_workspace_size(c["batch"], c["q_heads"], s["most"], s["top"])
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


def _own(s):
    c = s["case"]
    _handles(s)
    if c["op"] == "rope":
        return list(s["rope"].apply(s["positions"], s["q"], s["k"]))
    cache = s["cache"]
    if c["op"] == "rope_write":
        q = cache.rope_write(s["rope"], s["positions"], s["q"], s["k"], s["v"], s["slots"])
        if c["cache"] == "int8":
            return [q, *cache.gather(s["slots"])]
        return [q, s["pool"].view(torch.bfloat16 if c["cache"] == "bf16" else torch.float8_e4m3fn)]
    if c["op"] == "gather":
        return list(cache.gather(s["slots"]))
    if c["op"] == "tree":
        return [cache.tree_attention(s["q"], s["start"], s["most"], s["mask"], s["tables"], s["lens"], s["top"],
                                     out_dtype=s["q"].dtype, workspace=s["workspace"])]
    return [_whole_pool(s), cache.tree_commit(s["path"], s["accepted"], s["start"], s["tables"], s["lens"])]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "rope_write": _plain_rope_write, "gather": _plain_gather, "tree": _plain_tree,
            "commit": _plain_commit}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- work
def work(case):
    c = case
    D = c["dim"]
    if c["op"] in ("rope", "rope_write"):
        rows = c["q_heads"] + c["kv_heads"] * (1 if c["op"] == "rope" else 2)
        read = c["tokens"] * (rows * D * 2 + 4)
        wrote = c["tokens"] * (c["q_heads"] + (c["kv_heads"] if c["op"] == "rope" else 0)) * D * 2
        flops = 3 * c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["rot"]
        if c["op"] == "rope_write":
            bs, row, _ = _layout(c)
            wrote += c["tokens"] * c["kv_heads"] * (2 * row + (8 if c["cache"] == "int8" else 0))
            read += c["tokens"] * 4
            if c["cache"] == "int8":
                wrote += c["tokens"] * c["kv_heads"] * 2 * D * 2                 # the rows read back
        return {"bytes": read + wrote, "flops": flops}
    bs, row, rec = _layout(c)
    token = c["kv_heads"] * rec // bs                                            # one token's share of its records
    if c["op"] == "gather":
        return {"bytes": c["tokens"] * (token + 2 * c["kv_heads"] * D * 2 + 4), "flops": 2 * c["tokens"] * c["kv_heads"] * D}
    if c["op"] == "tree":
        n, size = (c["n_low"] + c["n_high"]) / 2, (c["l_low"] + c["l_high"]) / 2
        rows = c["batch"] * size * c["q_heads"]
        return {"bytes": c["batch"] * n * (token + 4 / 16) + rows * D * 4, "flops": 4 * rows * n * D}
    moved = c["batch"] * (c["accept"] + 1) / 2 * token
    return {"bytes": 2 * moved + c["batch"] * (4 * c["accept"] + 16), "flops": 0}


# ------------------------------------------------------------------------------- exact
def _turn64(x, positions, freqs, by, rot, layout):
    """The rotation as a product of complex numbers, 64 bits."""
    x = x.double()
    turn = torch.polar(torch.full_like(freqs, by), torch.zeros_like(freqs))[None]
    turn = turn * torch.exp(1j * (positions.double()[:, None] * freqs[None]))
    h = rot // 2
    pair = torch.complex(x[..., :h], x[..., h:rot]) if layout == "half" else torch.complex(x[..., 0:rot:2], x[..., 1:rot:2])
    pair = pair * turn[:, None]
    y = x.clone()
    if layout == "half":
        y[..., :h], y[..., h:rot] = pair.real, pair.imag
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = pair.real, pair.imag
    return y


def _e4m3_64(x):
    """The nearest E4M3 value (ties to even, largest 448), 64 bits."""
    mag = x.abs().clamp(max=448.0)
    exponent = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))).clamp(-6, 8)
    step = torch.exp2(exponent - 3)
    return torch.sign(x) * (torch.round(mag / step) * step).clamp(max=448.0)


def _rows64(s, blk, off):
    """K and V of cache rows (flat block and offset indexes), [rows][H][D] in 64 bits."""
    c = s["case"]
    bs, row, rec = _layout(c)
    H, D = c["kv_heads"], c["dim"]
    raw = s["pool"].view(-1, H, rec)[blk]                                        # [rows][H][record]
    i = torch.arange(blk.shape[0], device=blk.device)

    def part(first, count, width, dtype):
        t = raw[:, :, first:first + count * width].reshape(-1, H, count, width)[i, :, off].contiguous()
        return t.view(dtype)

    out = []
    for kv in range(2):
        code = part(kv * bs * row, bs, row, {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8, "int4": torch.uint8}[c["cache"]])
        if c["cache"] == "int4":
            code = torch.stack([code % 16, code // 16], -1).reshape(-1, H, D).double()
            if kv == 0:
                z = raw[:, :, 2 * bs * row:2 * bs * row + 4 * D].contiguous().view(torch.float16).double()
                out.append((code - z[..., D:]) * z[..., :D])
            else:
                z = part(2 * bs * row + 4 * D, bs, 4 * (D // _GROUP), torch.float16).double().view(-1, H, D // _GROUP, 2)
                out.append(((code.view(-1, H, D // _GROUP, _GROUP) - z[..., 1:]) * z[..., :1]).reshape(-1, H, D))
        elif c["cache"] == "int8":
            out.append(code.double() * part(2 * bs * row + 4 * bs * kv, bs, 4, torch.float32).double())
        elif c["cache"] == "fp8":
            out.append(code.double() * s["scale"][kv].double()[:, None])
        else:
            out.append(code.double())
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "commit" and c["cache"] != "bf16":
        return None                                                              # bytes only
    if c["op"] in ("rope", "rope_write"):
        how = (s["positions"], s["freqs"], s["by"], c["rot"], c["layout"])
        q, k = _turn64(s["q"], *how), _turn64(s["k"], *how)
    if c["op"] == "rope":
        return [q, k]
    if c["op"] == "rope_write":
        v = s["v"].double()
        if c["cache"] == "int8":
            back = []
            for x in (k, v):
                scale = (x.abs().amax(-1, keepdim=True) / 127).float().double()
                back.append(torch.round((x / scale).float().double()).clamp(-128, 127) * scale)
            return [q, *back]
        pool = s["pool"].view(torch.bfloat16 if c["cache"] == "bf16" else torch.float8_e4m3fn).double()
        bs, row, rec = _layout(c)
        n = 1 if c["cache"] == "fp8" else 2
        pool = pool.view(s["blocks"], c["kv_heads"], rec // n)
        blk, off = s["slots"].long() // bs, s["slots"].long() % bs
        for kv, x in enumerate((k, v)):
            if c["cache"] == "fp8":                          # the quotient is a binary32 by definition
                x = _e4m3_64((x / s["scale"][kv].double()[:, None]).float().double())
            pool[:, :, kv * bs * row // n:(kv + 1) * bs * row // n].unflatten(2, (bs, row // n))[blk, :, off] = x
        return [q, pool.reshape(-1)]
    if c["op"] == "gather":
        slots, bs = s["slots"].long(), _layout(c)[0]
        got = [_rows64(s, slots[i:i + 2048] // bs, slots[i:i + 2048] % bs) for i in range(0, len(slots), 2048)]
        return [torch.cat([g[0] for g in got]), torch.cat([g[1] for g in got])]
    if c["op"] == "commit":
        bs, row, rec = _layout(c)
        pool = s["pool"].view(torch.bfloat16).view(s["blocks"], c["kv_heads"], 2, bs, c["dim"]).clone()
        old, start, after = pool.clone(), s["start"].tolist(), []
        for b, (n, a) in enumerate(zip(s["lens"].tolist(), s["accepted"].tolist())):
            first = n - (start[b + 1] - start[b])
            table, path = s["tables"][b].tolist(), s["path"][b].tolist()
            for j in range(a):
                p, r = first + path[j], first + j
                pool[table[r // bs], :, :, r % bs] = old[table[p // bs], :, :, p % bs]
            after.append(first + a)
        return [pool.reshape(-1).double(), None]
    # tree: one sequence at a time, the visible positions of each query by the bits themselves
    H, D, g = c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    start, lens, out = s["start"].tolist(), s["lens"].tolist(), torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        k, v = (x.transpose(0, 1) for x in _rows64(s, s["tables"][b].long()[at // 16], at % 16))
        L = start[b + 1] - start[b]
        words = s["mask"][start[b]:start[b + 1]].long() % (1 << 32)
        see = torch.ones(L, n, dtype=torch.bool, device="cuda")
        for j in range(L):
            see[:, n - L + j] = (words[:, j // 32] // (1 << (j % 32))) % 2 == 1
        q = s["q"][start[b]:start[b + 1]].double().view(L, H, g, D)
        z = torch.einsum("lhgd,hnd->hgln", q, k) * D ** -0.5
        p = torch.softmax(z.masked_fill(~see, -math.inf), -1)
        out[start[b]:start[b + 1]] = torch.einsum("hgln,hnd->lhgd", p, v).reshape(L, H * g, D)
    return [out]
