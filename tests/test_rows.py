"""Cache rows by slot: kvq_gather (rows read back) and kvq_tree_commit (accepted rows moved).

A gathered value is one binary32 value rounded once to the activation type; the oracle's is the
same product (or difference and product) in float64, so they differ by half a step of the
activation type plus two binary32 roundings.  Commit moves bytes: exact."""

import ctypes

import numpy as np
import pytest
import torch

from quantized_paged_kv_02_b200 import inputs
from tests import helpers

helpers.ensure_built()
from quantized_paged_kv_02_b200 import kvq  # noqa: E402


def _desc(**kw):
    d = kvq.CacheDesc()
    base = dict(cache_dtype=3, act_dtype=0, scale_mode=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128,
                group_size=64, residual_len=128, residual_cap=192, max_seqs=1, pages=0x1000, residual=0x1000)
    base.update(kw)
    for k, v in base.items():
        setattr(d, k, v)
    return d


def test_gather_refusals():
    fake, odd, L = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004), kvq.lib
    call = lambda d=_desc(), s=fake, n=4, k=fake, v=fake: L.kvq_gather(ctypes.byref(d), s, n, k, v, None)
    assert call(n=0) == 0
    for bad in (dict(n=-1), dict(s=None), dict(k=None), dict(v=None), dict(k=odd), dict(v=odd), dict(d=_desc(pages=0))):
        assert call(**bad) == 1, bad
    assert call(d=_desc(head_dim=96)) == 2


def test_commit_refusals():
    fake, other, L = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x2000), kvq.lib

    def call(d=_desc(), path=fake, ma=4, acc=fake, B=2, qs=fake, bt=fake, mb=4, lens=fake, new=other):
        return L.kvq_tree_commit(ctypes.byref(d), path, ma, acc, B, qs, bt, mb, lens, new, None)

    assert call(B=0) == 0
    for bad in (dict(B=-1), dict(ma=-1), dict(path=None), dict(acc=None), dict(qs=None), dict(bt=None), dict(mb=0),
                dict(lens=None), dict(new=fake)):
        assert call(**bad) == 1, bad
    assert call(d=_desc(cache_dtype=5, scale_mode=4, block_size=64)) == 2


def test_commit_lengths_overlap_no_input():
    """new_lens is written while other CTAs of the same sequence may still read: no input, nor part of one."""
    at = dict(path=0x10000, acc=0x20000, qs=0x30000, bt=0x40000, lens=0x50000)
    size = dict(path=4 * 6 * 5, acc=24, qs=28, bt=4 * 6 * 7, lens=24)
    d, L = _desc(), kvq.lib

    def call(new):
        p = {k: ctypes.c_void_p(v) for k, v in at.items()}
        return L.kvq_tree_commit(ctypes.byref(d), p["path"], 5, p["acc"], 6, p["qs"], p["bt"], 7, p["lens"], ctypes.c_void_p(new), None)

    for name, base in at.items():
        for new in (base, base + 4, base - 20, base + size[name] - 4):
            assert call(new) == 1, (name, new - base)


# ------------------------------------------------------------------------------- GPU
gpu = pytest.mark.gpu
DENSE = [("int8", "per_token_head", 16, 128, "bf16"), ("int8", "per_token_head", 5, 64, "fp16"),
         ("int8", "per_channel", 16, 128, "bf16"), ("fp8", "per_head", 16, 128, "fp16"),
         ("fp8", "per_token_head", 7, 128, "bf16"), ("int8", "per_tensor", 16, 64, "bf16"),
         ("bf16", "none", 16, 128, "bf16"), ("fp16", "none", 3, 64, "fp16")]
LOW = [(cd, mode, 64, D, act) for cd in ("int4", "int2") for mode, D, act in
       (("kivi", 128, "bf16"), ("kivi_float_zero", 128, "fp16"), ("int4_per_token", 64, "bf16"))]


def _workload(cd, mode, bs, D, act, lens, seed=3, H=3):
    spec = inputs.Spec("rows", cd, act, mode, len(lens), H, H, D, bs, lens=lens, slack_blocks=2, seed=seed)
    return inputs.from_spec(spec)


@gpu
@pytest.mark.parametrize("cd,mode,bs,D,act", DENSE + LOW)
def test_gather_matches_oracle(cd, mode, bs, D, act):
    w = _workload(cd, mode, bs, D, act, [300, 1, 77])
    static = helpers.oracle_static_scales(w)
    oc, gc = helpers.oracle_cache(w, static), helpers.gpu_cache(w, static=static)
    paged = w.slot_mapping[w.slot_mapping >= 0]
    order = torch.randperm(paged.numel(), generator=torch.Generator().manual_seed(1))[:200]
    slots = torch.cat([paged[order], paged[order[:1]], torch.tensor([-1])]).int()      # one slot twice, one skipped
    k = torch.full((slots.numel(), 3, D), 7.0, dtype=inputs.act_torch_dtype(act), device="cuda")
    v = k.clone()
    gc.gather(slots.cuda(), k, v)
    eps = torch.finfo(k.dtype).eps / 2
    for i, s in enumerate(slots.tolist()):
        if s < 0:
            assert (k[i] == 7).all() and (v[i] == 7).all()
            continue
        want = oc.dequant_block(s // bs)[:, :, s % bs]
        for got, x in ((k[i], want[0]), (v[i], want[1])):
            assert (np.abs(helpers.np64(got) - x) <= eps * np.abs(x) + 2 * 2.0 ** -24 * 16 * np.abs(x).max() + 2.0 ** -25).all()
    assert gc.read_fault() == (0, 0)


@gpu
def test_gather_is_what_write_stored_and_counts_bad_slots():
    w = _workload("bf16", "none", 16, 128, "bf16", [50, 20])
    gc = helpers.gpu_cache(w)
    k, v = gc.gather(w.slot_mapping.cuda())
    assert torch.equal(k.cpu(), w.k) and torch.equal(v.cpu(), w.v)
    bad = torch.tensor([gc.num_blocks * 16, -2, int(w.slot_mapping[0])], dtype=torch.int32, device="cuda")
    k2 = torch.zeros((3, 3, 128), dtype=torch.bfloat16, device="cuda")
    gc.gather(bad, k2, k2.clone())
    assert (k2[:2] == 0).all() and torch.equal(k2[2].cpu(), w.k[0])
    assert gc.read_fault() == (2, 1)
    with pytest.raises(ValueError):
        gc.gather(bad, k2[:2], k2[:2])
    with pytest.raises(TypeError):
        gc.gather(bad, k2.half(), k2.half())


def _commit_reference(records, bs, off_v, row, off_s, tables, lens, starts, path, accepted):
    """Move rows of a copy of the records [NB][H][record], one sequence after another, reading
    everything before anything is written."""
    old, out, new = records.clone(), records.clone(), []
    for b, (n, a) in enumerate(zip(lens, accepted)):
        first = n - (starts[b + 1] - starts[b])
        for j in range(a):
            s, d = first + int(path[b][j]), first + j
            sb, so, db, do = int(tables[b][s // bs]), s % bs, int(tables[b][d // bs]), d % bs
            for base in (0, off_v):
                out[db, :, base + do * row:base + (do + 1) * row] = old[sb, :, base + so * row:base + (so + 1) * row]
            if off_s:
                for k in range(2):
                    at = off_s + 4 * bs * k
                    out[db, :, at + 4 * do:at + 4 * do + 4] = old[sb, :, at + 4 * so:at + 4 * so + 4]
        new.append(first + a)
    return out, new


@gpu
@pytest.mark.parametrize("cd,mode,bs,D,act", DENSE)
@pytest.mark.parametrize("H", [1, 5])
def test_commit_moves_the_accepted_rows(cd, mode, bs, D, act, H):
    sizes = [16, 1, 64, 300, 0, 5]
    lens = [200, 1, 64, 333, 9, 40]
    accepted = [6, 1, 64, 150, 0, 0]
    w = _workload(cd, mode, bs, D, act, lens, H=H)
    static = helpers.oracle_static_scales(w)
    gc = helpers.gpu_cache(w, static=static)
    g = torch.Generator().manual_seed(5)
    path = torch.zeros((6, 160), dtype=torch.int32)
    for b, (n, a) in enumerate(zip(sizes, accepted)):
        path[b, :a] = torch.randperm(n, generator=g)[:a].sort().values     # overlapping moves, many of them
        path[b, a:] = -9                                                   # not looked at
    starts = np.concatenate([[0], np.cumsum(sizes)])
    row = gc.desc.head_dim * (2 if cd in ("bf16", "fp16") else 1)
    want, new = _commit_reference(gc.records().cpu(), bs, bs * row, row, 2 * bs * row if mode == "per_token_head" else 0,
                                  w.block_tables, lens, starts, path, accepted)
    got = gc.tree_commit(path.cuda(), torch.tensor(accepted, dtype=torch.int32).cuda(),
                         torch.tensor(starts, dtype=torch.int32).cuda(), w.block_tables.cuda(), w.context_lens.cuda())
    assert got.tolist() == new
    assert torch.equal(gc.records().cpu(), want)
    assert gc.read_fault() == (0, 0)


@gpu
def test_commit_leaves_bad_paths_alone():
    """Each bad sequence is counted once and keeps its bytes and its length; the good one moves."""
    w = _workload("int8", "per_token_head", 16, 128, "bf16", [60] * 8, H=2)
    gc = helpers.gpu_cache(w)
    starts = torch.arange(9, dtype=torch.int32) * 10
    path = torch.tensor([[1, 4, 9], [4, 4, 5], [5, 3, 6], [0, 5, 10], [-1, 2, 3], [1, 2, 3], [1, 2, 3], [2, 5, 7]], dtype=torch.int32)
    accepted = torch.tensor([3, 3, 3, 3, 3, 4, -1, 3], dtype=torch.int32)
    tables = w.block_tables.clone()
    tables[7, 3] = gc.num_blocks                              # position 50 + 2 lies on it
    was = gc.records().cpu()
    want, new = _commit_reference(was, 16, 2048, 128, 4096, tables, [60] * 8, starts.tolist(), path, [3] + [0] * 7)
    got = gc.tree_commit(path.cuda(), accepted.cuda(), starts.cuda(), tables.cuda(), w.context_lens.cuda())
    assert got.tolist() == [53] + [60] * 7
    assert torch.equal(gc.records().cpu(), want)
    cnt, bits = gc.read_fault()
    assert cnt == 7 and bits == 64 | 4
    # an accepted count of 0 and no path at all
    none = torch.zeros((8, 0), dtype=torch.int32, device="cuda")
    got = gc.tree_commit(none, torch.zeros(8, dtype=torch.int32, device="cuda"), starts.cuda(), w.block_tables.cuda(), w.context_lens.cuda())
    assert got.tolist() == [50] * 8 and torch.equal(gc.records().cpu(), want)


@pytest.mark.gpu
def test_gather_and_commit_replay_in_a_graph_and_on_a_stream():
    """Captured once, replayed on other slots, paths and lengths; and the same calls on a stream of their own."""
    H, D, bs, B, L = 2, 128, 16, 3, 9
    g = torch.Generator().manual_seed(8)
    table = torch.randperm(24, generator=g)[:18].view(B, 6).int().cuda()
    rows = torch.randn((2, B * 90, H, D), generator=g).to(torch.bfloat16).cuda()
    every = (table.long()[:, torch.arange(90, device="cuda") // bs] * bs + torch.arange(90, device="cuda") % bs).int().reshape(-1)
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * L

    def fresh():
        c = kvq.PagedKVCache("int8", "bf16", "per_token_head", 24, bs, H, D)
        c.write(rows[0], rows[1], every)
        return c

    def draw(seed):
        r = torch.Generator().manual_seed(seed)
        acc = torch.randint(0, 6, (B,), generator=r)
        path = torch.stack([torch.randperm(L, generator=r)[:5].sort().values for _ in range(B)])
        lens = torch.randint(L, 90, (B,), generator=r)
        slots = every.cpu()[torch.randint(0, every.numel(), (40,), generator=r)]
        return [x.int().cuda() for x in (acc, path, lens, slots)]

    def direct(args, stream=None):
        c = fresh()
        acc, path, lens, slots = args
        torch.cuda.synchronize()
        new = c.tree_commit(path, acc, starts, table, lens, stream=stream)
        k, v = c.gather(slots, stream=stream)
        torch.cuda.synchronize()
        return new, k, v, c.pages.clone()

    c = fresh()
    acc, path, lens, slots = draw(0)
    new, k, v = torch.empty_like(lens), *(torch.empty((40, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.tree_commit(path, acc, starts, table, lens, new)
        c.gather(slots, k, v)
    for seed in (1, 2, 3):
        args = draw(seed)
        for at, x in zip((acc, path, lens, slots), args):
            at.copy_(x)
        c.pages.copy_(fresh().pages)
        graph.replay()
        torch.cuda.synchronize()
        for want in (direct(args), direct(args, torch.cuda.Stream())):
            assert all(torch.equal(a, b) for a, b in zip((new, k, v, c.pages), want))
    assert c.read_fault() == (0, 0)
