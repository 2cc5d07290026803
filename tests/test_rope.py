"""Rotary positions: kvq_rope and kvq_rope_write.

CPU: the oracle's pins (composition, norm, gradient), the library's host-only frequencies
against it, and the refusals.  GPU: values against the oracle.

Tolerances.  A rotated value y = m (a cos - b sin) is formed in binary32 from cosine and sine
rounded once (2^-24 each, times m): two products and one sum, each rounded once, so its error
is below 4 * 2^-24 * m (|a| + |b|); rounding to the activation type adds eps / 2 * |y|, half a
step at most (eps / 2 is 2^-8 for bf16 and 2^-11 for fp16)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp, quant, rope as oracle_rope
from tests import helpers

helpers.ensure_built()
from quantized_paged_kv_02_b200 import kvq  # noqa: E402

SCALINGS = {
    "none": {},
    "linear": {"factor": 4.0},
    "ntk": {"factor": 8.0},
    "wavelength": {"factor": 8.0, "original": 8192, "low": 1.0, "high": 4.0},
    "yarn": {"factor": 16.0, "original": 4096, "low": 1.0, "high": 32.0},
}


def _rope(dim, rot, layout="half", scaling="none", theta=500000.0, device="cuda", **kw):
    args = dict(SCALINGS[scaling])
    args["original_context"] = args.pop("original", 0)
    args.update(kw)
    return kvq.Rope(dim, rot, theta=theta, layout=layout, scaling=scaling, device=device, **args)


def _tolerance(x, y, rot, layout, m, eps):
    x = np.abs(x)
    a = x.copy()
    h = rot // 2
    if layout == "half":
        s = x[..., :h] + x[..., h:rot]
        a[..., :h], a[..., h:rot] = s, s
    else:
        s = x[..., 0:rot:2] + x[..., 1:rot:2]
        a[..., 0:rot:2], a[..., 1:rot:2] = s, s
    return 4 * 2.0 ** -24 * m * a + eps / 2 * np.abs(y) + 2.0 ** -40


# ------------------------------------------------------------------------------- CPU
def test_oracle_rotation_pins():
    g = np.random.default_rng(0)
    x = g.standard_normal((3, 2, 64))
    f, _ = oracle_rope.frequencies(32, 10000.0)
    for layout in ("half", "interleaved"):
        r = lambda v, t: oracle_rope.rotate(v, t, f, layout)
        assert np.array_equal(r(x, [0, 0, 0]), x)
        # turning by s then by t is turning by s + t, and back again is nothing
        assert np.abs(r(r(x, [5, 9, 100]), [7, -9, 1]) - r(x, [12, 0, 101])).max() < 1e-12
        # scores depend on the difference of positions only
        a = (r(x, [3, 3, 3])[0, 0] * r(x, [8, 8, 8])[1, 1]).sum()
        b = (r(x, [1003] * 3)[0, 0] * r(x, [1008] * 3)[1, 1]).sum()
        assert abs(a - b) < 1e-9
        # the rest of the head passes through
        assert np.array_equal(r(x, [4, 5, 6])[..., 32:], x[..., 32:])
    # an exact angle: one turn per 8 positions
    assert abs(oracle_rope.angle(10 ** 9 + 1, 2 * np.pi / 8) - np.pi / 4) < 1e-6
    assert oracle_rope.angle(2 ** 31 - 1, 1.0) == pytest.approx(np.angle(np.exp(1j * np.longdouble(2 ** 31 - 1))), abs=1e-6)


def test_rotation_gradient_is_the_rotation_backwards():
    """<r(x), w> has gradient r(w) at the negative positions: against differences."""
    g = np.random.default_rng(1)
    x, w = g.standard_normal((2, 1, 32)), g.standard_normal((2, 1, 32))
    f, _ = oracle_rope.frequencies(16, 1000.0)
    grad = oracle_rope.rotate(w, [-3, -70], f, "interleaved")
    for t in range(2):
        for d in range(0, 32, 5):
            e = np.zeros_like(x)
            e[t, 0, d] = 1e-6
            hi = (oracle_rope.rotate(x + e, [3, 70], f, "interleaved") * w).sum()
            lo = (oracle_rope.rotate(x - e, [3, 70], f, "interleaved") * w).sum()
            assert abs((hi - lo) / 2e-6 - grad[t, 0, d]) < 1e-8


@pytest.mark.parametrize("scaling", sorted(SCALINGS))
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_frequencies(scaling, rot):
    want, m = oracle_rope.frequencies(rot, 500000.0, scaling, **SCALINGS[scaling])
    r = _rope(128, rot, scaling=scaling, device="cpu")
    assert np.allclose(r.freqs.numpy(), want, rtol=1e-12, atol=0)
    assert r.attention_factor == pytest.approx(m, rel=1e-14)
    assert _rope(128, rot, scaling=scaling, device="cpu", attention_factor=0.5).attention_factor == 0.5


def test_scaled_frequencies_keep_the_fast_and_stretch_the_slow():
    plain, _ = oracle_rope.frequencies(128, 500000.0)
    for scaling in ("wavelength", "yarn"):
        kw = SCALINGS[scaling]
        f = _rope(128, 128, scaling=scaling, device="cpu").freqs.numpy()
        assert f[0] == plain[0] and f[-1] == pytest.approx(plain[-1] / kw["factor"], rel=1e-12)
        assert np.all(f <= plain * (1 + 1e-12)) and np.all(f >= plain / kw["factor"] * (1 - 1e-12))


def _bad_ropes():
    ok = dict(layout=0, rot_dim=64, scaling=0, original_context=0, theta=10000.0, factor=1.0, low=1.0, high=4.0,
              attention_factor=0.0)
    for name, change in {"layout": {"layout": 2}, "odd rot": {"rot_dim": 63}, "no rot": {"rot_dim": 0},
                         "scaling": {"scaling": 9}, "theta": {"theta": 0.0}, "theta nan": {"theta": float("nan")},
                         "factor": {"scaling": 1, "factor": 0.0}, "original": {"scaling": 3, "original_context": 0},
                         "low over high": {"scaling": 4, "original_context": 8, "low": 4.0, "high": 4.0},
                         "factor inf": {"scaling": 2, "factor": float("inf")},
                         "attention": {"attention_factor": -1.0}}.items():
        yield name, {**ok, **change}


@pytest.mark.parametrize("name,fields", list(_bad_ropes()))
def test_bad_rope_descriptors_are_refused(name, fields):
    r = kvq.RopeDesc()
    for k, v in fields.items():
        setattr(r, k, v)
    fake, L = ctypes.c_void_p(0x1000), kvq.lib
    assert L.kvq_rope_frequencies(ctypes.byref(r), None, None) == 1
    assert L.kvq_rope(ctypes.byref(r), fake, 0, 128, fake, 4, fake, 1024, 8, fake, 1024, None, 0, 0, None, 0, None) == 1


def test_rope_refusals():
    r = _rope(128, 64, device="cpu").desc
    fake, odd, L = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), kvq.lib

    def call(act=0, dim=128, pos=fake, T=4, q=fake, qs=1024, hq=8, qo=fake, qos=1024, k=None, ks=0, hk=0, ko=None, kos=0,
             freqs=fake, rope=r):
        return L.kvq_rope(ctypes.byref(rope), freqs, act, dim, pos, T, q, qs, hq, qo, qos, k, ks, hk, ko, kos, None)

    assert call(T=0) == 0 and call(hq=0) == 0                     # nothing to do
    for bad in (dict(act=2), dict(T=-1), dict(hq=-1), dict(q=None), dict(qo=None), dict(pos=None), dict(freqs=None),
                dict(q=odd), dict(qs=1020), dict(qs=512), dict(qos=1000), dict(k=None, hk=2), dict(dim=32)):
        assert call(**bad) == 1, bad                              # (dim 32: rot_dim 64 exceeds it)
    assert call(dim=96) == 2 and call(rope=_rope(128, 24, device="cpu").desc) == 2
    # rope_write: the same, and no low-bit cache
    d = kvq.CacheDesc()
    for k, v in dict(cache_dtype=3, act_dtype=0, scale_mode=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128,
                     pages=0x1000).items():
        setattr(d, k, v)

    def write(desc=d, T=4, k=fake, ks=256, v=fake, vs=256, slots=fake, hq=8, q=fake, qs=1024):
        return L.kvq_rope_write(ctypes.byref(desc), ctypes.byref(r), fake, fake, T, q, qs, hq, fake, 1024, k, ks, v, vs, slots, None)

    assert write(T=0) == 0
    for bad in (dict(k=None), dict(v=odd), dict(ks=128), dict(vs=252), dict(slots=None), dict(q=None), dict(hq=-1), dict(T=-2)):
        assert write(**bad) == 1, bad
    lo = kvq.CacheDesc()
    for k, v in dict(cache_dtype=5, act_dtype=0, scale_mode=4, num_blocks=8, block_size=64, num_kv_heads=2, head_dim=128,
                     group_size=64, residual_len=128, residual_cap=192, max_seqs=1, pages=0x1000, residual=0x1000).items():
        setattr(lo, k, v)
    assert write(desc=lo) == 2


def test_outputs_that_overlap_what_is_read_are_refused():
    """An output may be its own input; any other overlap (k read while q is rotated into it, one output over
    the other, shifted rows) would race.  Columns of one buffer do not overlap."""
    r, fake, L = _rope(128, 128, device="cpu").desc, ctypes.c_void_p(0x1000), kvq.lib
    P = lambda x: ctypes.c_void_p(x)
    A, B, C = 0x100000, 0x200000, 0x300000
    T = 5

    def rope(q, qs, qo, qos, k, ks, ko, kos):
        return L.kvq_rope(ctypes.byref(r), fake, 0, 128, fake, T, P(q), qs, 4, P(qo), qos, P(k), ks, 2, P(ko), kos, None)

    apart = 3 if not torch.cuda.is_available() else None            # (without a GPU the launch fails: KVQ_ERR_CUDA)
    row = 4 * 128 + 2 * 128                                         # q and k columns of one buffer
    for bad in ((A, 512, B, 512, B, 256, C, 256),                   # q_out over k
                (A, 512, A, 512, A, 512, B, 256),                   # in place over what is k too
                (A, 512, B, 512, C, 256, A + 16, 256),              # k_out inside q
                (A, 512, B, 512, C, 256, B + 2 * 512 * T - 16, 256),    # ... or in q_out's last bytes
                (A, 512, A + 256, 512, B, 256, C, 256),             # shifted
                (A, 512, A, 520, B, 256, C, 256),                   # another stride
                (A, row, A, row, A + 1008, row, A + 1008, row)):    # columns that share a chunk
        assert rope(*bad) == 1, bad
    if apart is not None:
        assert rope(A, row, A, row, A + 1024, row, A + 1024, row) == apart
        assert rope(A + 512, row, A + 512, row, A, row, A, row) == apart
        assert rope(A, 512, B, 512, A, 512, C, 256) == apart        # one tensor as both
        assert rope(A, 512, B, 512, C, 256, B + 2 * 512 * T, 256) == apart

    d = kvq.CacheDesc()
    for k, v in dict(cache_dtype=3, act_dtype=0, scale_mode=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128,
                     pages=0x900000).items():
        setattr(d, k, v)

    def write(q, qs, qo, qos, k, ks, v, vs):
        return L.kvq_rope_write(ctypes.byref(d), ctypes.byref(r), fake, fake, T, P(q), qs, 4, P(qo), qos, P(k), ks, P(v), vs, fake, None)

    for bad in ((A, 512, B, 512, B, 256, C, 256), (A, 512, B, 512, C, 256, B + 16, 256), (A, 512, A + 16, 512, B, 256, C, 256)):
        assert write(*bad) == 1, bad
    if apart is not None:
        fused = row + 256
        assert write(A, fused, A, fused, A + 1024, fused, A + 1536, fused) == apart
        assert write(A, 512, B, 512, C, 256, C, 256) == apart
    # rows read back: K and V apart
    assert L.kvq_gather(ctypes.byref(d), fake, 4, P(A), P(A), None) == 1
    assert L.kvq_gather(ctypes.byref(d), fake, 4, P(A), P(A + 4 * 512 - 16), None) == 1


# ------------------------------------------------------------------------------- GPU
gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _draw(T, heads, D, act, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, heads, D), generator=g).to(DT[act])


def _positions(T, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, 131072, (T,), generator=g, dtype=torch.int32)
    far = torch.tensor([0, 1, 2 ** 31 - 1, -5, 2 ** 24 + 1], dtype=torch.int32)
    p[:min(T, 5)] = far[:min(T, 5)]
    return p


@gpu
@pytest.mark.parametrize("T,hq,hk,D,rot,layout,scaling,act", [
    (1, 1, 1, 128, 128, "half", "none", "bf16"),
    (24, 64, 8, 128, 128, "half", "wavelength", "bf16"),
    (7, 5, 3, 64, 64, "interleaved", "linear", "fp16"),
    (33, 8, 2, 128, 32, "half", "yarn", "fp16"),
    (33, 8, 2, 128, 48, "interleaved", "ntk", "bf16"),
    (5, 3, 0, 64, 16, "half", "none", "fp16"),
    (300, 0, 4, 128, 96, "half", "yarn", "bf16"),
])
def test_rope_matches_oracle(T, hq, hk, D, rot, layout, scaling, act):
    r = _rope(D, rot, layout, scaling)
    pos = _positions(T, 3)
    q = _draw(T, hq, D, act, 1) if hq else None
    k = _draw(T, hk, D, act, 2) if hk else None
    got = r.apply(pos.cuda(), None if q is None else q.cuda(), None if k is None else k.cuda())
    f = r.freqs.cpu().numpy()
    for x, y in zip((q, k), got):
        if x is None:
            assert y is None
            continue
        n = min(T, 40)
        want = oracle_rope.rotate(helpers.np64(x[:n]), pos[:n].tolist(), f, layout, r.attention_factor)
        err = np.abs(helpers.np64(y[:n]) - want)
        assert (err <= _tolerance(helpers.np64(x[:n]), want, rot, layout, r.attention_factor, torch.finfo(DT[act]).eps)).all()
        assert torch.equal(y.cpu()[..., rot:], x[..., rot:])       # the rest of the head, bit for bit


@gpu
@pytest.mark.parametrize("exponent", [24, 28, 31])
@pytest.mark.parametrize("pair", [0, 1])
def test_far_angles_keep_binary32_accuracy(exponent, pair):
    """Pairs (a, b) = (1, 1) turned to where one half almost vanishes: what is left of a - b is the
    angle's error and those of cosine and sine, which the 16-bit output resolves.  The angle is good to
    binary64, so the bound is that of cosine, sine (half a step of values up to 1: 2^-25 each), one product's
    rounding (2^-25) and the output's."""
    r = _rope(128, 16, "half", theta=500000.0)
    f = float(r.freqs[pair])
    top = 2 ** exponent - 1
    t = np.arange(top - 4000000, top + 1, dtype=np.int64)
    turns = t.astype(np.longdouble) * np.longdouble(f) / (2 * np.longdouble("3.14159265358979323846264338327950288"))
    near = np.abs(turns - np.floor(turns) - np.longdouble(0.125))           # an eighth of a turn: cos = sin
    t = t[np.argsort(near)[:24]]
    x = torch.zeros(24, 1, 128, dtype=torch.bfloat16)
    x[:, 0, pair] = x[:, 0, 8 + pair] = 1.0
    y = r.apply(torch.from_numpy(t.astype(np.int32)).cuda(), x.cuda())[0].cpu().double().numpy()[:, 0, pair]
    ang = np.array([oracle_rope.angle(int(p), f) for p in t])
    want = np.cos(ang) - np.sin(ang)
    assert np.abs(want).max() < 2.0 ** -14                                   # (of the positions: near enough)
    err = np.abs(y - want)
    assert (err <= 3 * 2.0 ** -25 + 2.0 ** -8 * np.abs(want)).all(), float(err.max())


@gpu
def test_rope_takes_fused_rows_in_place_and_gaps():
    """Views into fused projection rows, rotated in place: v and the gap are left alone."""
    r = _rope(128, 128)
    T, hq, hk = 19, 6, 2
    buf = _draw(T, hq + 2 * hk + 1, 128, "bf16", 5).cuda()
    was = buf.clone()
    pos = _positions(T, 6).cuda()
    q, k = buf[:, :hq], buf[:, hq:hq + hk]
    want = r.apply(pos, q.contiguous(), k.contiguous())
    r.apply(pos, q, k, q_out=q, k_out=k)
    assert torch.equal(buf[:, :hq], want[0]) and torch.equal(buf[:, hq:hq + hk], want[1])
    assert torch.equal(buf[:, hq + hk:], was[:, hq + hk:])
    # backwards again: the rotation undone, up to two roundings of each element
    back = r.apply(-pos.long().clamp(max=2 ** 31 - 1).int(), want[0])[0]
    x = was[:, :hq].float()
    pair = x.abs() + x.abs().roll(64, -1)
    assert ((back.float() - x).abs() <= 2 * 2.0 ** -8 * 1.5 * pair + 1e-6).all()


@gpu
def test_rope_wrapper_checks():
    r = _rope(128, 128)
    q, pos = _draw(4, 2, 128, "bf16", 1).cuda(), torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        r.apply(pos[:3], q)
    with pytest.raises(TypeError):
        r.apply(pos.long(), q)
    with pytest.raises(ValueError):
        r.apply(pos, q.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(TypeError):
        r.apply(pos, q, q.half())
    with pytest.raises(ValueError):
        r.apply(pos, q, q_out=q[:, :1])
    with pytest.raises(TypeError):
        r.apply(pos, q.float())
    for bad in ((pos.cpu(), q), (pos, q.cpu()), (pos,)):            # host tensors, nothing to rotate
        with pytest.raises(ValueError):
            r.apply(*bad)
    for freqs in (r.freqs[:-1], r.freqs.float()):
        with pytest.raises(ValueError):
            kvq.kvq_rope(r.desc, freqs, pos, q)
    a, b = r.apply(pos, q, q)                                       # one tensor as both
    assert torch.equal(a, b) and torch.equal(a, r.apply(pos, q)[0])


def _cache(cd, act, mode, nb, bs, H, D, seed=0):
    sk = sv = None
    if mode in ("per_head", "per_tensor", "per_channel"):
        n = {"per_head": (H,), "per_tensor": (1,), "per_channel": (H, D)}[mode]
        g = torch.Generator().manual_seed(seed)
        top = 127 if cd == "int8" else 448
        sk, sv = (torch.rand(n, generator=g) + 3.5) / top, (torch.rand(n, generator=g) + 3.5) / top
    return kvq.PagedKVCache(cd, act, mode, nb, bs, H, D, static_k_scale=sk, static_v_scale=sv)


def _k_codes(c, slots):
    """K codes [T, H, D] and per-token scales [T, H] of the listed slots."""
    bs, H, D = c.block_size, c.num_kv_heads, c.head_dim
    rec = c.records().cpu()
    blk, off = slots.long() // bs, slots.long() % bs
    codes = rec[:, :, :bs * D].reshape(c.num_blocks, H, bs, D)[blk, :, off]
    s = None
    if c.scale_mode == "per_token_head":
        s = rec[:, :, 2 * bs * D:2 * bs * D + 4 * bs].contiguous().view(torch.float32)[blk, :, off]
    return codes.numpy(), None if s is None else s.numpy()


@gpu
@pytest.mark.parametrize("cd,mode,bs,D,act,layout,rot,T", [
    ("int8", "per_token_head", 16, 128, "bf16", "half", 128, 50),
    ("int8", "per_token_head", 5, 64, "fp16", "interleaved", 64, 33),
    ("int8", "per_head", 16, 128, "fp16", "half", 64, 1),
    ("int8", "per_channel", 16, 128, "bf16", "interleaved", 96, 17),
    ("fp8", "per_head", 16, 128, "bf16", "half", 128, 64),
    ("fp8", "per_token_head", 32, 64, "bf16", "half", 32, 20),
    ("fp8", "per_tensor", 16, 128, "bf16", "interleaved", 128, 9),
])
def test_rope_write_quantizes_the_rotated_rows(cd, mode, bs, D, act, layout, rot, T):
    H, hq = 3, 6
    r = _rope(D, rot, layout, "yarn")
    nb = -(-T // bs) + 3
    c = _cache(cd, act, mode, nb, bs, H, D)
    ref = _cache(cd, act, mode, nb, bs, H, D)
    q, k, v = _draw(T, hq, D, act, 1), _draw(T, H, D, act, 2), _draw(T, H, D, act, 3)
    if T > 3:
        k[2], v[3] = 0, 0                                          # all-zero rows: scale 0
    pos = _positions(T, 4)
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(7))[:T].int()
    if T > 4:
        slots[4] = -1                                              # not stored
    got = c.rope_write(r, pos.cuda(), q.cuda(), k.cuda(), v.cuda(), slots.cuda())
    want_q = r.apply(pos.cuda(), q.cuda())[0]
    assert torch.equal(got, want_q)
    # V rows as kvq_write stores them; everything not written keeps the fill byte
    ref.write(k.cuda(), v.cuda(), slots.cuda())
    row = D
    a, b = c.records().cpu(), ref.records().cpu()
    assert torch.equal(a[:, :, bs * row:2 * bs * row], b[:, :, bs * row:2 * bs * row])
    if mode == "per_token_head":
        o = 2 * bs * row + 4 * bs
        assert torch.equal(a[:, :, o:], b[:, :, o:])
    live = slots >= 0
    free = torch.ones(nb * bs, dtype=torch.bool)
    free[slots[live].long()] = False
    kept = a[:, :, :bs * row].reshape(nb, H, bs, row).permute(0, 2, 1, 3).reshape(nb * bs, H, row)[free]
    assert (kept == 0x5A).all()
    # K codes: those of the exact rotated value, or of one within its binary32 error of it
    f = r.freqs.cpu().numpy()
    x = oracle_rope.rotate(helpers.np64(k), pos.tolist(), f, layout, r.attention_factor)
    tol = _tolerance(helpers.np64(k), x, rot, layout, r.attention_factor, 0.0)
    codes, scales = _k_codes(c, slots[live])
    x, tol = x[live.numpy()], tol[live.numpy()]
    top = 127.0 if cd == "int8" else 448.0
    if mode == "per_token_head":
        s = scales.astype(np.float64)
        amax = np.abs(x).max(-1)
        assert (np.abs(s - amax / top) <= (tol.max(-1) + 2.0 ** -24 * amax) / top + 1e-45).all()
        s = s[..., None]
    else:
        s = np.asarray(c.k_scales.cpu().numpy()[:{"per_head": H, "per_tensor": 1, "per_channel": H * D}[mode]], np.float64)
        s = {"per_head": lambda: s[None, :, None], "per_tensor": lambda: s[None, None], "per_channel": lambda: s.reshape(1, H, D)}[mode]()
    s = np.broadcast_to(s, x.shape).astype(np.float32)

    def code(y):
        y = y.astype(np.float32)
        return quant.int8_quantize(y, s) if cd == "int8" else quant.fp8_quantize(y, s)

    def value(cc):
        return np.asarray(cc).view(np.int8).astype(np.float64) if cd == "int8" else fp.e4m3_decode(np.asarray(cc, np.uint8))

    have, lo, hi = value(codes.view(np.uint8)), value(np.asarray(code(x - 2 * tol)).astype(np.int8 if cd == "int8" else np.uint8)), \
        value(np.asarray(code(x + 2 * tol)).astype(np.int8 if cd == "int8" else np.uint8))
    assert ((have >= np.minimum(lo, hi)) & (have <= np.maximum(lo, hi))).all()
    assert c.read_fault() == (0, 0)


@gpu
@pytest.mark.parametrize("act,layout", [("bf16", "half"), ("fp16", "interleaved")])
def test_rope_write_to_16_bit_cache_is_rope_then_write(act, layout):
    T, H, hq, D = 40, 2, 4, 128
    r = _rope(D, 64, layout, "linear")
    a, b = _cache(act, act, "none", 6, 16, H, D), _cache(act, act, "none", 6, 16, H, D)
    buf = _draw(T, hq + 2 * H, D, act, 1).cuda()
    q, k, v = buf[:, :hq], buf[:, hq:hq + H], buf[:, hq + H:]
    pos = _positions(T, 2).cuda()
    slots = torch.randperm(96, generator=torch.Generator().manual_seed(1))[:T].int().cuda()
    got = a.rope_write(r, pos, q, k, v, slots)
    want = r.apply(pos, q, k)
    b.write(want[1], v.contiguous(), slots)
    assert torch.equal(got, want[0]) and torch.equal(a.pages, b.pages)
    # without q, and with a bad slot: counted, the rest stored
    slots[0] = 96
    assert a.rope_write(r, pos, None, k, v, slots) is None
    assert a.read_fault() == (1, 1)


@gpu
def test_rope_write_replays_in_a_graph_and_on_a_stream():
    T, H, hq, D = 24, 8, 64, 128
    r = _rope(D, 128)
    c = _cache("int8", "bf16", "per_token_head", 8, 16, H, D)
    q, k, v = (_draw(T, h, D, "bf16", s).cuda() for h, s in ((hq, 1), (H, 2), (H, 3)))
    pos, slots = _positions(T, 4).cuda(), torch.arange(T, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    c.rope_write(r, pos, q, k, v, slots, q_out=out)
    want, pages = out.clone(), c.pages.clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        c.rope_write(r, pos, q, k, v, slots, q_out=out)
    out.zero_()
    c.pages.fill_(0x5A)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(c.pages, pages)
