"""kvq_tree_attention (drafted trees over the cache) against the float64 oracle.

Tolerance.  With float32 output a result o = sum w v / sum w carries the errors of its weights:
a score is a binary32 sum of 128 products whose magnitudes add up to S (in units of the base-2
exponent, at most about 60 for these inputs), so it is off by at most 128 * 2^-24 * S < 5e-4,
which moves the result by no more than 2 * 5e-4 * ln 2 of spread = sum w |v| / sum w; the
weights' own rounding (two halves: 2^-16 at worst) adds less than 2^-15 of it.  Together
below 2^-10 spread.  bf16 output rounds once more (eps / 2 = 2^-8 of the result, half a step
at most) and, for 8-bit and fp16 caches, weights of 11 bits (2^-11 of spread, inside the 2^-10).
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle import attention
from quantized_paged_kv_02_b200 import inputs
from tests import helpers

helpers.ensure_built()
from quantized_paged_kv_02_b200 import kvq  # noqa: E402


# ------------------------------------------------------------------------------- helpers
def random_tree(size, g, chain=0.4):
    """sees[i]: drafted indexes token i sees (itself and its ancestors)."""
    sees = []
    for i in range(size):
        up = []
        if i:
            p = i - 1 if torch.rand((), generator=g) < chain else int(torch.randint(0, i, (), generator=g))
            up = sees[p]
        sees.append(up + [i])
    return sees


def pack(sees, words):
    m = np.zeros((len(sees), words), np.uint32)
    for i, s in enumerate(sees):
        for j in s:
            m[i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    return torch.from_numpy(m.view(np.int32).copy())


def make(cd, mode, act, hq, hk, D, bs, lens, sizes, seed=1, outliers="", empty=(), noise=False):
    """A workload with a drafted tree per sequence; rows listed in `empty` see no drafted token,
    with noise every row sees a random set."""
    spec = inputs.Spec("tree", cd, act, mode, len(lens), hq, hk, D, bs, lens=lens, slack_blocks=3, seed=seed, outliers=outliers)
    w = inputs.from_spec(spec)
    g = torch.Generator().manual_seed(seed + 100)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32)
    q = torch.randn((int(starts[-1]), hq, D), generator=g).to(inputs.act_torch_dtype(act))
    sees = []
    for s in sizes:
        t = random_tree(s, g)
        if noise:
            t = [torch.nonzero(torch.rand(s, generator=g) < 0.5).flatten().tolist() for _ in range(s)]
        sees += t
    for i in empty:
        sees[i] = []
    most = max(max(sizes), 1)
    return w, q, starts, sees, pack(sees, (most + 31) // 32), most


def run(gc, w, q, starts, mask, most, out_dtype=torch.float32, **kw):
    return gc.tree_attention(q.cuda(), starts.cuda(), most, mask.cuda(), w.block_tables.cuda(), w.context_lens.cuda(),
                             max(w.max_context, 1), out_dtype=out_dtype, **kw)


def check(got, want, spread, out_dtype):
    eps = 0.0 if out_dtype == torch.float32 else torch.finfo(out_dtype).eps / 2
    err = np.abs(helpers.np64(got) - want)
    tol = 2.0 ** -10 * spread + eps * np.abs(want) + 1e-7
    assert (err <= tol).all(), float((err / tol).max())


# ------------------------------------------------------------------------------- CPU
def test_oracle_tree_pins():
    """A chain is chunked prefill; a row that sees only itself of the draft is decode of a
    cache without the others; a row that sees nothing gives zeros."""
    w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 4, 2, 64, 16, [40, 9], [5, 9])
    oc = helpers.oracle_cache(w)
    args = (w.block_tables.numpy(), w.context_lens.numpy())
    chain = [list(range(i + 1)) for i in range(5)] + [list(range(i + 1)) for i in range(9)]
    a, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), chain, *args)
    b = attention.prefill_attention(oc, helpers.np64(q), starts.numpy(), *args)
    assert np.abs(a - b).max() < 1e-12 and (spread >= np.abs(a) - 1e-12).all()
    one, _ = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), [[]] * 14, *args)
    n = np.array([35, 0])
    assert np.abs(one[3] - attention.decode_attention(oc, helpers.np64(q[[3, 3]]), args[0], n)[0]).max() < 1e-12
    assert not one[5:].any()                                   # no prefix, no bit


def test_mask_words_hold_the_bits():
    sees = random_tree(70, torch.Generator().manual_seed(2))
    m = pack(sees, 3).numpy().view(np.uint32)
    for i, s in enumerate(sees):
        assert [j for j in range(96) if (int(m[i, j // 32]) >> (j % 32)) & 1] == sorted(s)


def test_output_type_is_checked():
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        kvq.kvq_tree_attention(_desc(), q, None, 2, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32),
                               torch.zeros(1, dtype=torch.int32), 64, q.double())


def _desc(**kw):
    d = kvq.CacheDesc()
    base = dict(cache_dtype=3, act_dtype=0, scale_mode=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128,
                group_size=64, residual_len=128, residual_cap=192, max_seqs=1, pages=0x1000, residual=0x1000,
                k_scales=0x1000, v_scales=0x1000)
    base.update(kw)
    for k, v in base.items():
        setattr(d, k, v)
    return d


def test_workspace_size():
    size = kvq.kvq_tree_workspace_size
    # tensor cores: two partial tiles of 128 rows per CTA, each row 128 floats, (offset, sum)
    assert size(_desc(), 4, 16, 8, 1000) == 2 * 148 * 128 * (128 + 2) * 4
    assert size(_desc(), 4, 16, 8, 1000) == size(_desc(), 64, 16, 1024, 10 ** 6)
    # CUDA cores: a short context has one split and needs none
    assert size(_desc(head_dim=64), 1, 4, 2, 32) == 0
    a = size(_desc(head_dim=64), 1, 4, 2, 8192)
    assert a > 0 and a == size(_desc(head_dim=64), 1, 4, 2, 8192)
    for bad, want in ((dict(cache_dtype=5, scale_mode=4, block_size=64), 2), (dict(head_dim=96), 2), (dict(num_blocks=0), 1)):
        with pytest.raises(kvq.KVQError) as e:
            size(_desc(**bad), 1, 4, 2, 64)
        assert e.value.status == want
    with pytest.raises(kvq.KVQError):
        size(_desc(), 1, 5, 2, 64)
    with pytest.raises(kvq.KVQError) as e:
        size(_desc(), 1, 4, 1025, 64)
    assert e.value.status == 2


def test_tree_refusals():
    fake, odd, L = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), kvq.lib
    need = kvq.kvq_tree_workspace_size(_desc(), 2, 4, 8, 64)

    def call(d=_desc(), q=fake, T=8, B=2, hq=4, qs=fake, mt=8, mask=fake, mw=1, bt=fake, mb=4, lens=fake, mc=64, scale=0.0,
             out=fake, od=2, ws=fake, wsb=need):
        return L.kvq_tree_attention(ctypes.byref(d), q, T, B, hq, qs, mt, mask, mw, bt, mb, lens, mc, ctypes.c_float(scale), out, od,
                                    ws, wsb, None)

    assert call(B=0) == 0 and call(T=0) == 0 and call(mt=0) == 0
    for bad in (dict(T=-1), dict(B=-1), dict(hq=3), dict(hq=0), dict(mt=-1), dict(mt=33), dict(mb=0), dict(mc=-1), dict(od=3),
                dict(scale=-1.0), dict(scale=float("nan")), dict(q=None), dict(q=odd), dict(out=odd), dict(out=None), dict(qs=None),
                dict(mask=None), dict(bt=None), dict(lens=None), dict(ws=None), dict(wsb=need - 1), dict(ws=odd),
                dict(d=_desc(pages=0))):
        assert call(**bad) == 1, bad
    assert call(mt=1025, mw=33) == 2
    assert call(mc=1 << 30, B=8) == 2                            # more blocks than the schedule can count
    assert call(d=_desc(cache_dtype=6, scale_mode=4, block_size=64)) == 2
    # the CUDA-core kernel's partials are per query row: more rows than batch * max_tree do not fit
    d = _desc(head_dim=64)
    assert call(d=d, T=17, mc=8192, mb=512, wsb=1 << 30) == 1


# ------------------------------------------------------------------------------- GPU
gpu = pytest.mark.gpu
F32, B16, H16 = torch.float32, torch.bfloat16, torch.float16

CASES = {
    # one token, one position; no prefix at all; a tail behind a block; several blocks
    "int8": ("int8", "per_token_head", "bf16", 16, 2, 128, 16, [1, 7, 140, 517, 1000], [1, 7, 13, 16, 3], F32),
    "int8-bf16out": ("int8", "per_token_head", "bf16", 16, 2, 128, 16, [1, 7, 140, 517, 1000], [1, 7, 13, 16, 3], B16),
    "int8-fp16": ("int8", "per_token_head", "fp16", 4, 2, 128, 16, [256, 129], [64, 40], H16),
    "int8-static": ("int8", "per_head", "bf16", 8, 2, 128, 16, [300, 200], [20, 5], B16),
    "int8-tensor": ("int8", "per_tensor", "fp16", 3, 1, 128, 16, [128, 127], [43, 1], F32),
    "fp8": ("fp8", "per_head", "bf16", 8, 2, 128, 16, [300, 31, 700], [32, 31, 33], B16),
    "fp8-token": ("fp8", "per_token_head", "bf16", 5, 1, 128, 16, [400, 60], [27, 60], F32),
    "bf16": ("bf16", "none", "bf16", 16, 2, 128, 16, [64, 512, 385], [64, 1, 17], B16),
    "bf16-f32": ("bf16", "none", "bf16", 8, 8, 128, 16, [200, 90], [90, 33], F32),
    "fp16": ("fp16", "none", "fp16", 7, 1, 128, 16, [260, 130], [19, 130], H16),
    "fp16-bf16out": ("fp16", "none", "fp16", 2, 2, 128, 16, [260, 130], [140, 130], B16),
    # groups wider than 8, several tiles of rows, heads that straddle tiles
    "g16": ("int8", "per_token_head", "bf16", 16, 1, 128, 16, [300, 77], [37, 9], F32),
    "g6": ("fp8", "per_tensor", "bf16", 6, 1, 128, 16, [333], [100], F32),
    # no sequence has a query, and one of three has
    "none": ("int8", "per_token_head", "bf16", 4, 2, 128, 16, [50, 20], [0, 0], F32),
    "one-of-three": ("int8", "per_token_head", "bf16", 4, 2, 128, 16, [50, 20, 300], [0, 3, 0], F32),
    # CUDA cores: head_dim 64, other block sizes, per-channel scales, splits
    "d64": ("int8", "per_token_head", "fp16", 8, 4, 64, 16, [128, 77], [9, 33], F32),
    "d64-long": ("fp8", "per_head", "bf16", 2, 1, 64, 16, [2000], [5], B16),
    "bs5": ("int8", "per_token_head", "bf16", 4, 2, 128, 5, [99, 6], [12, 6], F32),
    "bs32-bf16": ("bf16", "none", "bf16", 6, 2, 128, 32, [70, 33], [7, 33], F32),
    "channel": ("int8", "per_channel", "bf16", 8, 2, 128, 16, [150, 40], [10, 3], F32),
}


@gpu
@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("noise", [False, True])
def test_tree_matches_oracle(name, noise):
    cd, mode, act, hq, hk, D, bs, lens, sizes, od = CASES[name]
    empty = [0] if sizes[0] else []
    w, q, starts, sees, mask, most = make(cd, mode, act, hq, hk, D, bs, lens, sizes, empty=empty, noise=noise)
    static = helpers.oracle_static_scales(w)
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    got = run(gc, w, q, starts, mask, most, od)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    check(got, want, spread, od)
    assert gc.read_fault() == (0, 0)


@gpu
def test_outlier_channels():
    w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 8, 2, 128, 16, [600, 300], [16, 9], outliers="kv")
    oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    for od in (F32, B16):
        check(run(gc, w, q, starts, mask, most, od), want, spread, od)


@gpu
@pytest.mark.parametrize("cd,mode,act", [("int8", "per_token_head", "bf16"), ("fp8", "per_head", "fp16"), ("bf16", "none", "bf16")])
@pytest.mark.parametrize("step", [0.3, 4.0])
def test_scores_that_keep_growing(cd, mode, act, step):
    """Keys along the query's direction, longer with every position: each block holds a new maximum, by a
    little or by many powers of two, so that the running maximum is re-based in visible blocks."""
    n, L, D = 700, 4, 128
    w, q, starts, sees, mask, most = make(cd, mode, act, 4, 1, D, 16, [n], [L], seed=3)
    d = torch.randn(D, generator=torch.Generator().manual_seed(9))
    d = d / d.norm()
    q = (q.float() * 0.02 + 4.0 * d).to(q.dtype)
    grow = torch.arange(n).float()[:, None, None] * step / 64
    w.k = (w.k.float() * 0.05 + grow * d).to(w.k.dtype)
    w.v = (w.v.float() * (1 + torch.arange(n).float()[:, None, None] / 100)).to(w.v.dtype)     # V scales grow too
    static = None if mode != "per_head" else ([0.25], [0.125])
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    for od in (F32, B16):
        check(run(gc, w, q, starts, mask, most, od), want, spread, od)
    # and shrinking: the maximum comes first
    w.k, w.v = w.k.flip(0).contiguous(), w.v.flip(0).contiguous()
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    check(run(gc, w, q, starts, mask, most), want, spread, F32)


@gpu
@pytest.mark.parametrize("cd,mode,act", [("int8", "per_token_head", "fp16"), ("fp8", "per_head", "bf16"), ("bf16", "none", "bf16")])
@pytest.mark.parametrize("up", [12.0, 60.0, 400.0])
def test_one_position_far_above_the_rest(cd, mode, act, up):
    """One visible position whose score is `up` powers of two above all before it: its weight relative to
    the running maximum overflows a half (12), or binary32 (400: scores of 2^8 carry an error of
    128 * 2^-24 * 400 = 2^-8.4, but then no other weight is above 2^-300 and the result is that V row)."""
    n, L, D = 500, 3, 128
    w, q, starts, sees, mask, most = make(cd, mode, act, 4, 1, D, 16, [n], [L], seed=4)
    d = torch.randn(D, generator=torch.Generator().manual_seed(9)).sign() / D ** 0.5
    q = (q.float() * 0.01 + 8.0 * d).to(q.dtype)
    w.k = (w.k.float() * 0.05).to(w.k.dtype)
    w.k[333] += (d * (up / (8.0 * 1.4426950408889634) * D ** 0.5)).to(w.k.dtype)
    static = None if mode != "per_head" else ([0.0625], [0.03125])
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    for od in (F32, B16):
        check(run(gc, w, q, starts, mask, most, od), want, spread, od)


@gpu
def test_scores_of_minus_infinity_and_vanishing_queries():
    """A prefix whose scores overflow to -inf weighs nothing; q next to 0 weighs every position alike."""
    w, q, starts, sees, mask, most = make("bf16", "none", "bf16", 4, 1, 128, 16, [300, 90], [3, 90], seed=6)
    q = q.abs() + 4
    w.k[:150] = -1e38                                           # (all of the first blocks, of both streams)
    oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())

    check(run(gc, w, q, starts, mask, most), want, spread, F32)
    w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 4, 1, 128, 16, [300], [3], seed=6)
    q = (q.float() * 1e-37).to(torch.bfloat16)
    oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    check(run(gc, w, q, starts, mask, most), want, spread, F32)


@gpu
def test_largest_trees():
    """1024 drafted tokens, once without any prefix: 64 tiles of rows per head, walked by groups of CTAs,
    beside a sequence whose last tile row has one tile."""
    w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 16, 2, 128, 16, [1024, 1500, 300], [1024, 1024, 70],
                                          noise=True)
    oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    got = run(gc, w, q, starts, mask, most)
    check(got, want, spread, F32)
    assert torch.equal(got, run(gc, w, q, starts, mask, most))


@gpu
def test_bounds_need_not_be_tight():
    """max_tree and max_context are upper bounds: the largest ones change no result."""
    for D, bs, cd in ((128, 16, "int8"), (64, 16, "int8"), (128, 32, "bf16")):
        mode = "none" if cd == "bf16" else "per_token_head"
        lens = [1 + i % 60 for i in range(300)]
        w, q, starts, sees, mask, most = make(cd, mode, "bf16", 2, 2, D, bs, lens, [1 + i % 2 if n > 1 else 1 for i, n in enumerate(lens)])
        gc = helpers.gpu_cache(w)
        a = (q.cuda(), starts.cuda())
        b = (mask.cuda(), w.block_tables.cuda(), w.context_lens.cuda())
        want = gc.tree_attention(*a, most, *b, w.max_context)
        # (the tensor-core kernel's schedule counts fewer than 2^27 blocks)
        far = 2 ** 31 - 1 if D == 64 or bs != 16 else 2 ** 32 // (300 * 2) // 64 * 64 - 64
        for most_, context in ((32, w.max_context), (most, far), (32, far)):
            got = gc.tree_attention(*a, most_, *b, context)
            assert (got - want).abs().max().item() <= 2.0 ** -18 * max(1.0, want.abs().max().item())
        assert gc.read_fault() == (0, 0)


@gpu
def test_sequences_that_share_pages():
    """Two sequences with one prefix in the same pages."""
    w, q, starts, sees, mask, most = make("fp8", "per_token_head", "bf16", 8, 2, 128, 16, [300, 300], [12, 12])
    w.block_tables[1, :18] = w.block_tables[0, :18]
    oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    check(run(gc, w, q, starts, mask, most), want, spread, F32)


@gpu
def test_many_short_sequences_and_one_long():
    """Several units per CTA, and one unit cut into hundreds of parts."""
    lens = [1 + 7 * (i % 40) for i in range(200)] + [20000]
    sizes = [min(n, 1 + i % 5) for i, n in enumerate(lens)]
    w, q, starts, sees, mask, most = make("fp8", "per_head", "bf16", 8, 2, 128, 16, lens, sizes)
    static = helpers.oracle_static_scales(w)
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    got = run(gc, w, q, starts, mask, most)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    check(got, want, spread, F32)
    # the same call again, bit for bit
    assert torch.equal(got, run(gc, w, q, starts, mask, most))


@gpu
def test_one_token_that_sees_itself_is_decode():
    w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 16, 2, 128, 16, [1000, 517, 33], [1, 1, 1])
    gc = helpers.gpu_cache(w)
    dec = gc.decode(q.cuda(), w.block_tables.cuda(), w.context_lens.cuda(), w.max_context)
    assert (run(gc, w, q, starts, mask, most) - dec).abs().max().item() <= 1e-4


@gpu
@pytest.mark.parametrize("D", [128, 64])
def test_rejected_sequences_and_rows_of_nobody(D):
    w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 4, 2, D, 16, [60, 50, 3, 40], [5, 4, 3, 8])
    gc = helpers.gpu_cache(w)
    q = torch.cat([q, q[:3]])                                   # rows behind the last sequence
    mask = torch.cat([mask, mask[:3]])
    lens = w.context_lens.clone()
    lens[1], lens[2] = 10 ** 6, 2                                # beyond max_context; fewer positions than drafted
    out = torch.full((q.shape[0], 4, D), 7.0, device="cuda")
    ws = torch.empty(kvq.kvq_tree_workspace_size(gc.desc, 4, 4, 8, 64) + 16, dtype=torch.uint8, device="cuda")
    kvq.kvq_tree_attention(gc.desc, q.cuda(), starts.cuda(), 7, mask.cuda(), w.block_tables.cuda(), lens.cuda(), 64, out, ws)
    cnt, bits = gc.read_fault()
    assert cnt == 3 and bits == 4                                # (the fourth drafts 8 > 7)
    assert (out[5:] == 7).all() and (out[:5] != 7).all()


@gpu
@pytest.mark.parametrize("cd,mode,D", [("int8", "per_token_head", 128), ("fp8", "per_head", 128), ("bf16", "none", 128),
                                       ("bf16", "none", 64)])
def test_bad_block_ids_are_left_out(cd, mode, D):
    """Positions on a bad page count as absent: the result is that of a mask without them."""
    w, q, starts, sees, mask, most = make(cd, mode, "bf16", 4, 2, D, 16, [400, 60], [9, 4])
    static = helpers.oracle_static_scales(w)
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    tables = w.block_tables.clone()
    tables[0, 3], tables[0, 20], tables[1, 0] = -1, gc.num_blocks, 10 ** 9
    got = gc.tree_attention(q.cuda(), starts.cuda(), most, mask.cuda(), tables.cuda(), w.context_lens.cuda(), w.max_context)
    cnt, bits = gc.read_fault()
    assert cnt >= 3 and bits == 2
    K, V = zip(*(oc.gather(w.block_tables[b].numpy(), int(w.context_lens[b])) for b in range(2)))
    qd = helpers.np64(q)
    for b, gone in ((0, set(range(48, 64)) | set(range(320, 336))), (1, set(range(16)))):
        n, L = int(w.context_lens[b]), int(starts[b + 1] - starts[b])
        for i in range(L):
            row = int(starts[b]) + i
            at = [p for p in list(range(n - L)) + [n - L + j for j in sees[row]] if p not in gone]
            for h in range(4):
                o = attention.softmax_attention(qd[row, h], K[b][h // 2][at], V[b][h // 2][at], D ** -0.5)
                spread = attention.softmax_attention(qd[row, h], K[b][h // 2][at], np.abs(V[b][h // 2][at]), D ** -0.5)
                assert (np.abs(helpers.np64(got[row, h]) - o) <= 2.0 ** -10 * spread + 1e-7).all()


@gpu
@pytest.mark.parametrize("cd,mode,D", [("bf16", "none", 128), ("fp8", "per_head", 128), ("int8", "per_token_head", 128),
                                       ("fp8", "per_token_head", 128), ("bf16", "none", 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_drafted_rows_reach_only_those_that_see_them(cd, mode, D, value):
    """K and V of drafted token 2 and of stale rows behind the context hold NaN or infinities.  Rows
    that do not see token 2 are those of a clean cache, bit for bit; V's reach the others."""
    n, L = 150, 9
    w, q, starts, sees, mask, most = make(cd, mode, "bf16", 4, 1, D, 16, [n], [L])
    static = helpers.oracle_static_scales(w)
    clean, dirty = helpers.gpu_cache(w, static=static), helpers.gpu_cache(w, static=static)
    pos = n - L + 2
    slot = lambda p: int(w.block_tables[0, p // 16]) * 16 + p % 16
    k, v = w.k[pos:pos + 1].clone(), w.v[pos:pos + 1].clone()
    v[:, :, 3] = value
    if value != value:
        k[:, :, 5] = value
    stale = torch.full_like(w.k[:1], value)
    dirty.write(k.cuda(), v.cuda(), torch.tensor([slot(pos)], dtype=torch.int32, device="cuda"))
    for p in range(n, -(-n // 16) * 16):
        dirty.write(stale.cuda(), stale.cuda(), torch.tensor([slot(p)], dtype=torch.int32, device="cuda"))
    a, b = run(clean, w, q, starts, mask, most), run(dirty, w, q, starts, mask, most)
    blind = [i for i in range(L) if 2 not in sees[i]]
    seeing = [i for i in range(L) if 2 in sees[i]]
    assert blind and seeing
    assert torch.equal(a[blind], b[blind])
    # what the cache holds of the row (an INT8 or FP8 writer may have made it finite) reaches the rest:
    # a NaN in K every channel, an unusable V channel its own
    kg, vg = (x[0, 0] for x in dirty.gather(torch.tensor([slot(pos)], dtype=torch.int32, device="cuda")))
    if torch.isnan(kg).any():
        assert torch.isnan(b[seeing]).all()
    else:
        assert torch.equal(torch.isfinite(b[seeing]), torch.isfinite(vg).expand(len(seeing), 4, D))
    if cd == "bf16":
        assert not torch.isfinite(vg[3])


def crowd(gc, w, q, sees, od, copies=300):
    """One sequence's tree `copies` times over the same pages, so that most CTAs hold whole units: every
    copy's output, [copies, L, Hq, D]."""
    L = q.shape[0]
    out = gc.tree_attention(q.repeat(copies, 1, 1).cuda(), (torch.arange(copies + 1, dtype=torch.int32) * L).cuda(), L,
                            pack(sees, (L + 31) // 32).repeat(copies, 1).cuda(), w.block_tables.repeat(copies, 1).cuda(),
                            w.context_lens.repeat(copies).cuda(), w.max_context, out_dtype=od)
    return out.view(copies, *q.shape)


def hide(sees, starts, b, j):
    """No query of sequence b sees its drafted token j."""
    for i in range(int(starts[b]), int(starts[b + 1])):
        sees[i] = [t for t in sees[i] if t != j]


@gpu
@pytest.mark.parametrize("cd,act,od", [("int8", "bf16", B16), ("int8", "fp16", F32), ("fp8", "bf16", F32), ("fp8", "bf16", B16)])
@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 14, 2.0 ** 20, 1e30])
def test_hidden_drafted_rows_of_any_size_reach_nobody(cd, act, od, ratio):
    """Drafted rows that no query sees hold V `ratio` times the others' (per-token scales): the result is
    that of the rows which are seen."""
    if act == "fp16" and ratio > 2.0 ** 12:
        ratio = 2.0 ** 12 if ratio < 2.0 ** 20 else 2.0 ** 14      # (65504 is the largest V that fp16 holds)
    lens, sizes = [140, 64, 700], [13, 64, 9]
    w, q, starts, sees, mask, most = make(cd, "per_token_head", act, 8, 2, 128, 16, lens, sizes)
    for b, j in ((0, 4), (1, 0), (1, 63), (2, 8)):
        hide(sees, starts, b, j)
        row = int(w.seq_start[b]) + lens[b] - sizes[b] + j
        w.v[row] = (w.v[row].float().clamp(-3.9, 3.9) * ratio).to(w.v.dtype)
    mask = pack(sees, mask.shape[1])
    oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    check(run(gc, w, q, starts, mask, most, od), want, spread, od)


@gpu
@pytest.mark.parametrize("cd,od", [("int8", B16), ("int8", F32), ("fp8", B16), ("fp8", F32)])
@pytest.mark.parametrize("fill", [0x5A, 0xDA, 0xFF, 0x7F, 0x00])
def test_padding_that_was_never_written(cd, od, fill):
    """A tree padded to a fixed size whose padding went to slot -1 and is masked for everyone: its K, V and
    scales are whatever the page held (1.5e16, -3e16, NaN, 3.4e38, 0)."""
    lens, sizes = [140, 64, 33], [40, 64, 7]
    w, q, starts, sees, mask, most = make(cd, "per_token_head", "bf16", 8, 2, 128, 16, lens, sizes)
    for b, pad in ((0, 15), (1, 40), (2, 2)):
        for j in range(sizes[b] - pad, sizes[b]):
            hide(sees, starts, b, j)
            w.slot_mapping[int(w.seq_start[b]) + lens[b] - sizes[b] + j] = -1
    mask = pack(sees, mask.shape[1])
    oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w, fill=fill)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    check(run(gc, w, q, starts, mask, most, od), want, spread, od)
    assert gc.read_fault() == (0, 0)


@gpu
@pytest.mark.parametrize("cd,od", [("int8", B16), ("int8", F32), ("fp8", B16), ("fp8", F32)])
@pytest.mark.parametrize("at,ratio", [(5, 2.0 ** 12), (5, 2.0 ** 16), (5, 1e30), (333, 2.0 ** 16), (333, 1e30), (580, 1e30)])
def test_large_values_of_no_weight(cd, od, at, ratio):
    """A visible position of the prefix whose V is `ratio` times the others' and whose score lies 200 powers
    of two below theirs weighs nothing, and takes no bits from those that do."""
    n, L, D = 600, 4, 128
    w, q, starts, sees, mask, most = make(cd, "per_token_head", "bf16", 4, 1, D, 16, [n], [L], seed=7)
    d = torch.randn(D, generator=torch.Generator().manual_seed(9)).sign() / D ** 0.5
    q = (q.float() * 0.01 + 8.0 * d).to(q.dtype)
    w.k[at] = (-d * 200).to(w.k.dtype)
    w.v[at] = (w.v[at].float() * ratio).to(w.v.dtype)
    oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    check(crowd(gc, w, q, sees, od), want, spread, od)


@gpu
@pytest.mark.parametrize("low,high", [(-84, 0), (0, 84), (-84, 84)])
def test_value_scales_of_every_size(low, high):
    """V of one size in the first half of the context and of another in the second, in either order: the ends
    of the range that the header names."""
    n, L = 800, 5
    for a, b in ((low, high), (high, low)):
        w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 4, 1, 128, 16, [n], [L], seed=8)
        size = torch.where(torch.arange(n) < n // 2, 2.0 ** (a + 7), 2.0 ** (b + 5)).view(n, 1, 1)
        w.v = (w.v.float() * size).to(w.v.dtype)
        oc, gc = helpers.oracle_cache(w), helpers.gpu_cache(w)
        want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
        for od in (F32, B16):
            check(crowd(gc, w, q, sees, od), want, spread, od)


@gpu
@pytest.mark.parametrize("cd,mode,act", [("int8", "per_token_head", "bf16"), ("int8", "per_head", "bf16"), ("fp8", "per_head", "fp16"),
                                         ("fp16", "none", "fp16"), ("bf16", "none", "bf16")])
@pytest.mark.parametrize("gap", [14, 18, 22, 30])
@pytest.mark.parametrize("at", [0, 2000])
def test_a_sink_of_no_value(cd, mode, act, gap, at):
    """One position of nearly all the weight whose V is 0, and 4000 others 2^gap below it with one sign in V:
    the result is what those say, so their weights' roundings add up instead of cancelling."""
    n, L, D = 4000, 3, 128
    w, q, starts, sees, mask, most = make(cd, mode, act, 2, 1, D, 16, [n], [L], seed=11)
    d = torch.randn(D, generator=torch.Generator().manual_seed(9)).sign() / D ** 0.5
    q = (0.0 * q.float() + 8.0 * d).to(q.dtype)
    unit = D ** 0.5 / (8.0 * 1.4426950408889634)                   # a key d * unit * x scores x (base-2 units)
    w.k[:] = (d * unit * 0.4).to(w.k.dtype)
    w.k[at] = (d * unit * (gap + 0.4)).to(w.k.dtype)
    w.v = (1 + 0.1 * w.v.float().clamp(-4, 4)).to(w.v.dtype)
    w.v[at] = 0
    static = helpers.oracle_static_scales(w)
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    for od in (F32, B16):
        got = crowd(gc, w, q, sees, od)
        # the absolute part of the bound: 2^-31 of the largest weight per position, where scales are not per token
        # and the others lie more than 2^18 below it
        floor = 2.0 ** -31 * n * 1.5 / (1 + n * 2.0 ** -gap) if gap > 18 and (mode == "per_head" or cd == "fp16") else 0.0
        eps = 0.0 if od == F32 else torch.finfo(od).eps / 2
        err = np.abs(helpers.np64(got) - want)
        assert (err <= 2.0 ** -10 * spread + eps * np.abs(want) + floor).all(), float((err / spread).max())


@gpu
@pytest.mark.parametrize("cd,mode,act", [("int8", "per_token_head", "bf16"), ("fp8", "per_head", "bf16"), ("bf16", "none", "bf16")])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 36, 1e30])
def test_scores_beyond_an_exponents_range(cd, mode, act, size):
    """Scores whose last binary32 bit is worth many powers of two: the largest one's V row is the result.  A
    score is off by at most 128 * 2^-24 of the magnitudes that it sums, so rows are checked whose largest lies
    further above the rest than twice that (and by more than 64 powers of two)."""
    n, L = 330, 3
    w, q, starts, sees, mask, most = make(cd, mode, act, 4, 1, 128, 16, [n], [L], seed=14)
    q = (q.float() * size).to(q.dtype)
    static = helpers.oracle_static_scales(w)
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    K = oc.gather(w.block_tables[0].numpy(), n)[0][0]
    clear = np.zeros((L, 4), bool)
    for i in range(L):
        at = list(range(n - L)) + [n - L + j for j in sees[i]]
        for h in range(4):
            z = np.sort(K[at] @ helpers.np64(q[i, h])) * 128 ** -0.5
            off = 128 * 2.0 ** -24 * (np.abs(K[at]) @ np.abs(helpers.np64(q[i, h]))).max() * 128 ** -0.5
            clear[i, h] = z[-1] - z[-2] > 2 * off + 64
    assert clear.sum() >= 8
    for od in (F32, B16):
        got = run(gc, w, q, starts, mask, most, od)
        assert torch.isfinite(got).all()
        check(got[torch.from_numpy(clear).to(got.device)], want[clear], spread[clear], od)


@gpu
@pytest.mark.parametrize("cd,mode", [("int8", "per_token_head"), ("fp8", "per_token_head"), ("fp8", "per_head"), ("int8", "per_tensor"),
                                     ("bf16", "none")])
@pytest.mark.parametrize("kind", ["large", "inf", "nan", "steps"])
def test_queries_do_not_reach_each_other(cd, mode, kind):
    """One tile of query rows (tokens and heads) holds rows of very different size, or one with an infinity or
    a NaN: every other row's result is its own."""
    L, hq = 12, 4
    w, q, starts, sees, mask, most = make(cd, mode, "bf16", hq, 1, 128, 16, [500], [L], seed=12)
    w.k[:, :, 9] = 0                                                 # (a channel where a query may be anything)
    bad = []
    if kind == "large":
        q[3, 1] *= 1e30
        bad = [(3, 1)]                                               # (scores of 1e30: some one position's V)
    elif kind == "steps":                                            # 2^-2 .. 2^-60 of the first
        q = (q.float() * 2.0 ** (-torch.arange(L).float() * 5 - 2).view(L, 1, 1)).to(q.dtype)
        q[0, 2] *= 16
    else:
        q[3, 1, 7] = float(kind)
        q[5, 0, 9] = 2.0 ** 20
        bad = [(3, 1)]
    static = helpers.oracle_static_scales(w)
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    clean = q.clone()
    clean[3, 1] = 0 if kind in ("inf", "nan") else clean[3, 1]
    want, spread = attention.tree_attention(oc, helpers.np64(clean), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    rest = np.ones((L, hq), bool)
    for at in bad:
        rest[at] = False
    for od in (F32, B16):
        got = run(gc, w, q, starts, mask, most, od)
        check(got[torch.from_numpy(rest).to(got.device)], want[rest], spread[rest], od)
        if kind == "large":
            assert torch.isfinite(got).all()


@gpu
@pytest.mark.parametrize("cd,mode,act", [("int8", "per_head", "bf16"), ("fp8", "per_head", "fp16"), ("fp16", "none", "fp16")])
@pytest.mark.parametrize("drafted", [False, True])
def test_a_new_maximum_in_the_second_half_of_a_block(cd, mode, act, drafted):
    """32 positions, and 2^26 above them one of no value in the same block's second half: the first ones'
    probabilities, already stored, are scaled by 2^-26 or so, less than the smallest fp16, to what is more."""
    gap, D = 26, 128
    n, L = (60, 60) if drafted else (64, 0)
    n += 0 if drafted else 3
    L = L or 3
    w, q, starts, sees, mask, most = make(cd, mode, act, 2, 1, D, 16, [n], [L], seed=15)
    d = torch.randn(D, generator=torch.Generator().manual_seed(9)).sign() / D ** 0.5
    q = (0.0 * q.float() + 8.0 * d).to(q.dtype)
    unit = D ** 0.5 / (8.0 * 1.4426950408889634)
    w.k[:] = (d * unit * 0.4).to(w.k.dtype)
    w.k[40] = (d * unit * (gap + 0.4)).to(w.k.dtype)
    w.v = (1 + 0.1 * w.v.float().clamp(-4, 4)).to(w.v.dtype)
    w.v[40] = 0
    sees = [list(range(L)) if drafted else s for s in sees]
    mask = pack(sees, mask.shape[1])
    static = helpers.oracle_static_scales(w)
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    want, spread = attention.tree_attention(oc, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    for od in (F32, B16):
        got = run(gc, w, q, starts, mask, most, od)
        err = np.abs(helpers.np64(got) - want)
        # 2^-31 of the largest probability (which is 1) per position, as far as fp16 goes
        eps = 0.0 if od == F32 else torch.finfo(od).eps / 2
        assert (err <= 2.0 ** -10 * spread + eps * np.abs(want) + 2.0 ** -31 * n * 1.5).all(), float((err / spread).max())


@gpu
@pytest.mark.parametrize("od", [F32, B16])
def test_an_infinity_of_the_prefix_stays_in_its_channel(od):
    """V of a visible prefix position holds an infinity: its channel is infinite or NaN, the others are as they
    would be without it."""
    w, q, starts, sees, mask, most = make("bf16", "none", "bf16", 8, 2, 128, 16, [500, 90], [9, 9])
    clean = helpers.oracle_cache(w)
    want, spread = attention.tree_attention(clean, helpers.np64(q), starts.numpy(), sees, w.block_tables.numpy(), w.context_lens.numpy())
    w.v[100, 0, 7], w.v[int(w.seq_start[1]) + 3, 1, 64] = float("inf"), float("-inf")
    got = run(helpers.gpu_cache(w), w, q, starts, mask, most, od)
    hit = np.zeros(got.shape, bool)
    hit[:9, :4, 7] = hit[9:, 4:, 64] = True
    assert not torch.isfinite(got[torch.from_numpy(hit).cuda()]).any()
    check(got[torch.from_numpy(~hit).cuda()], want[~hit], spread[~hit], od)


@gpu
def test_two_streams_graph_and_backgrounds():
    """Two calls at once with workspaces of their own, and a captured one replayed on other inputs."""
    w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 16, 2, 128, 16, [3000, 1200, 64], [16, 3, 9])
    gc = helpers.gpu_cache(w)
    args = (starts.cuda(), most, mask.cuda(), w.block_tables.cuda(), w.context_lens.cuda(), w.max_context)
    q1 = q.cuda()
    q2 = torch.randn_like(q1)
    want1, want2 = gc.tree_attention(q1, *args), gc.tree_attention(q2, *args)
    n = gc.tree_workspace_size(3, 16, most, w.max_context)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(want1) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, x, o, k in zip(streams, (q1, q2), outs, ws):
            gc.tree_attention(x, *args, out=o, workspace=k, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want1) and torch.equal(outs[1], want2)
    buf, out = q1.clone(), torch.empty_like(want1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gc.tree_attention(buf, *args, out=out, workspace=ws[0])
    for x, want in ((q2, want2), (q1, want1)):
        buf.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@gpu
def test_workspace_of_a_call_on_another_stream_is_not_handed_out():
    """The call's own workspace and output belong to its stream: what the current stream allocates and
    fills meanwhile is other memory."""
    w, q, starts, sees, mask, most = make("fp8", "per_head", "bf16", 8, 2, 128, 16, [3000, 2500], [16, 9])
    gc = helpers.gpu_cache(w, static=helpers.oracle_static_scales(w))
    args = (q.cuda(), starts.cuda(), most, mask.cuda(), w.block_tables.cuda(), w.context_lens.cuda(), w.max_context)
    want = gc.tree_attention(*args)
    n = gc.tree_workspace_size(2, 8, most, w.max_context)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s):
            torch.cuda._sleep(100000)
        got = gc.tree_attention(*args, stream=s)
        for _ in range(20):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@gpu
def test_draft_verify_and_commit():
    """A run of the operators as a serving step uses them: the drafted rows rotated by their depth and
    written, the tree attended, its accepted path committed, and the next decode step equal to
    that of a cache to which the accepted tokens were written one after another."""
    H, hq, D, n0, L = 2, 8, 128, 200, 12
    g = torch.Generator().manual_seed(3)
    rope = kvq.Rope(D, 128, theta=500000.0)
    caches = [kvq.PagedKVCache("int8", "bf16", "per_token_head", 20, 16, H, D) for _ in range(2)]
    table = torch.randperm(20, generator=g)[:14].int()[None]
    slot = lambda p: (table[0, p // 16] * 16 + p % 16).int()
    rows = lambda T, h: torch.randn((T, h, D), generator=g).to(torch.bfloat16).cuda()
    pk, pv, pq = rows(n0, H), rows(n0, H), rows(n0, hq)
    for c in caches:
        c.rope_write(rope, torch.arange(n0, dtype=torch.int32).cuda(), pq, pk, pv, slot(torch.arange(n0)).cuda())
    sees = random_tree(L, g)
    path = max(sees, key=len)
    dk, dv, dq = rows(L, H), rows(L, H), rows(L, hq)
    depth = torch.tensor([n0 + len(s) - 1 for s in sees], dtype=torch.int32).cuda()
    spec, plain = caches
    q = spec.rope_write(rope, depth, dq, dk, dv, slot(torch.arange(n0, n0 + L)).cuda())
    starts = torch.tensor([0, L], dtype=torch.int32).cuda()
    lens = torch.tensor([n0 + L], dtype=torch.int32).cuda()
    tree = spec.tree_attention(q, starts, L, pack(sees, 1).cuda(), table.cuda(), lens, n0 + L)
    acc = torch.tensor([len(path)], dtype=torch.int32).cuda()
    new = spec.tree_commit(torch.tensor([path], dtype=torch.int32).cuda(), acc, starts, table.cuda(), lens)
    assert new.tolist() == [n0 + len(path)]
    # the accepted tokens one at a time: the tree's row is the step's output, and the caches agree
    for j, t in enumerate(path):
        at = torch.tensor([n0 + j], dtype=torch.int32).cuda()
        qj = plain.rope_write(rope, at, dq[t:t + 1], dk[t:t + 1], dv[t:t + 1], slot(torch.tensor([n0 + j])).cuda())
        assert torch.equal(qj[0], q[t])
        step = plain.decode(qj, table.cuda(), at + 1, n0 + L)
        assert (step[0] - tree[t]).abs().max().item() <= 2e-3
    got = [c.gather(slot(torch.arange(n0 + len(path))).cuda()) for c in caches]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@gpu
def test_wrapper_checks():
    w, q, starts, sees, mask, most = make("int8", "per_token_head", "bf16", 4, 2, 128, 16, [60], [5])
    gc = helpers.gpu_cache(w)
    a = dict(q=q.cuda(), q_start=starts.cuda(), max_tree=most, tree_mask=mask.cuda(), block_tables=w.block_tables.cuda(),
             context_lens=w.context_lens.cuda(), max_context=64)
    for bad in (dict(q=a["q"].half()), dict(tree_mask=a["tree_mask"][:3]), dict(context_lens=a["context_lens"].repeat(2)),
                dict(block_tables=a["block_tables"][0]), dict(q=a["q"].transpose(1, 2))):
        with pytest.raises(ValueError):
            gc.tree_attention(**{**a, **bad})
    for bad in (dict(tree_mask=a["tree_mask"].long()), dict(q_start=a["q_start"].long())):
        with pytest.raises(TypeError):
            gc.tree_attention(**{**a, **bad})
    cold = kvq.PagedKVCache("int8", "bf16", "per_token_head", gc.num_blocks, 16, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        cold.tree_attention(**a)
    # a host tensor is refused, not dereferenced
    for name in ("q", "q_start", "tree_mask", "block_tables", "context_lens"):
        with pytest.raises(ValueError):
            gc.tree_attention(**{**a, name: a[name].cpu(), "out": torch.empty_like(a["q"])})
