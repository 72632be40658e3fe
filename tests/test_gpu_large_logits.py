"""Queries and keys of 1e4 to 1e6: finite logits of 2^30 and more in log2 units,
whose rounding is wider than any weight's exponent. Where a row's largest logit
is ahead of the next by more than both may be off, the definition gives its
value alone; every other row stays finite. (The packed and the 4-bit calls have
such tests beside their others.)"""
import math

import numpy as np
import pytest
import torch

from oracle.cache_ops import bf16_round

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = [3e4, 1e5, 1e6]


@pytest.fixture(scope="module")
def resa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_quest_b200 as m
    return m


def rnd(seed, *shape, size=1.0):
    x = np.random.Generator(np.random.PCG64(seed)).standard_normal(shape).astype(np.float32)
    return bf16_round(bf16_round(x) * np.float32(size))


def dev(x, dtype="bf16"):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(DT[dtype])


def clear_rows(q, k, scale, seen):
    """q [n, d], k [m, d], seen [n, m]: the rows whose largest logit is ahead by
    more than fp32 may be off, and where it is. Any order of fp32 additions of d
    products errs by (d + 8) 2^-24 of their magnitudes at most, truncated ones
    by twice that; the rounding to log2 units adds its own."""
    z = np.where(seen, q.astype(np.float64) @ k.astype(np.float64).T * scale, -np.inf)
    mags = np.abs(q).astype(np.float64) @ np.abs(k).astype(np.float64).T * scale
    e = (2 * q.shape[-1] + 32) * 2.0 ** -24 * np.where(seen, mags, 0).max(-1)
    top = np.sort(z, -1)
    gap = np.full(len(z), np.inf)
    two = np.isfinite(top[:, -2])
    gap[two] = top[two, -1] - top[two, -2]
    return np.flatnonzero(gap > 2 * e + 100), z.argmax(-1)


def check(out, v, rows, arg, dtype):
    """out [n, d]: v's row arg[i] alone in rows `rows`, rounded once; finite elsewhere."""
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
    assert np.isfinite(out).all()
    for i in rows:
        want = v[arg[i]].astype(np.float64)
        assert (np.abs(out[i] - want) <= half * 1.02 * np.abs(want)).all(), i
    return len(rows)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("G", [1, 4])
def test_prefill(resa, size, G):
    B, H, n, d, cap = 2, 2, 330, 128, 336
    q, k, v = rnd(1, B, n, H * G, d, size=size), rnd(2, B, H, cap, d, size=size), rnd(3, B, H, cap, d)
    qt, kt, vt = dev(q), dev(k), dev(v)
    desc = torch.zeros(B, H, cap // 16, 2, d, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(qt)
    ws = resa.alloc_workspace(resa.dims_for(kt, H * G), cap)
    scale = 1.0 / math.sqrt(d)
    resa.prefill(qt, kt, vt, desc, n, scale, out, ws)
    assert resa.workspace_status(ws) == resa.RESA_OK
    o, seen, clear = out.double().cpu().numpy(), np.tril(np.ones((n, n), bool)), 0
    for b in range(B):
        for h in range(H * G):
            rows, arg = clear_rows(q[b, :, h], k[b, h // G, :n], scale, seen)
            clear += check(o[b, :, h], v[b, h // G], rows, arg, "bf16")
    assert clear > B * H * G * n // 2


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("n", [200, 5000])                 # (one split; several, merged)
@pytest.mark.parametrize("ragged", [False, True])
def test_rectify(resa, size, n, ragged):
    B, H, G, f, d = 2, 2, 4, 32, 128
    cap = (n + 15) // 16 * 16
    q, k, v = rnd(1, B, f, H * G, d, size=size), rnd(2, B, H, cap, d, size=size), rnd(3, B, H, cap, d)
    kt, vt, qt = dev(k), dev(v), dev(q)
    lens = [n, n - 7 if ragged else n]
    kf = np.stack([k[b, :, x - f:x].transpose(1, 0, 2) for b, x in enumerate(lens)])
    vf = np.stack([v[b, :, x - f:x].transpose(1, 0, 2) for b, x in enumerate(lens)])
    desc = torch.zeros(B, H, cap // 16, 2, d, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(qt)
    ws = resa.alloc_workspace(resa.dims_for(kt, H * G), cap, f=f)
    scale = 1.0 / math.sqrt(d)
    if ragged:
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        resa.rectify_varlen(qt, dev(kf), dev(vf), kt, vt, desc, lt, n, f, scale, out, ws)
    else:
        resa.rectify(qt, dev(kf), dev(vf), kt, vt, desc, n, f, scale, out, ws)
    assert resa.workspace_status(ws) == resa.RESA_OK
    o, clear = out.double().cpu().numpy(), 0
    for b, x in enumerate(lens):
        seen = np.arange(x)[None] <= (x - f + np.arange(f))[:, None]
        for h in range(H * G):
            rows, arg = clear_rows(q[b, :, h], k[b, h // G, :x], scale, seen)
            clear += check(o[b, :, h], v[b, h // G], rows, arg, "bf16")
    assert clear > B * H * G * f // 2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("form", ["dense", "blocks", "weights"])
def test_decode(resa, dtype, size, form):
    B, H, G, d, n = 2, 4, 8, 128, 700
    q, k, v = rnd(1, B, H * G, d, size=size), rnd(2, B, H, 704, d, size=size), rnd(3, B, H, 704, d)
    kt, vt, qt = dev(k, dtype), dev(v, dtype), dev(q, dtype)
    out = torch.zeros_like(qt)
    dims, scale = resa.dims_for(kt, H * G), 1.0 / math.sqrt(d)
    ws = resa.alloc_weights_workspace(dims, n)
    w = torch.zeros(B, H, 704, device="cuda")
    if form == "dense":
        resa.decode_dense(qt, None, None, kt, vt, None, n, scale, out, ws)
    elif form == "blocks":
        sel = torch.arange(44, dtype=torch.int32, device="cuda").expand(B, H, -1).contiguous()
        resa.attend_blocks(qt, kt, vt, n, sel, scale, out, ws)
    else:
        resa.decode_dense_weights(qt, None, None, kt, vt, None, w, n, scale, out, None, ws)
    assert resa.workspace_status(ws) == resa.RESA_OK
    o, wn, clear = out.double().cpu().numpy(), w.double().cpu().numpy(), 0
    for b in range(B):
        for g in range(H):
            hs = slice(g * G, g * G + G)
            rows, arg = clear_rows(q[b, hs], k[b, g, :n], scale, np.ones((G, n), bool))
            clear += check(o[b, hs], v[b, g], rows, arg, dtype)
            if form == "weights" and len(rows) == G:
                assert np.array_equal(wn[b, g, :n], np.bincount(arg, minlength=n))
    assert clear > B * H * G // 2
