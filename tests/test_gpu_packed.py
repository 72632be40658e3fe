"""Packed prompts on the GPU against the plain causal attention of each
sequence (oracle/cache_ops.py), in 64 bits."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def resa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_quest_b200 as m
    return m


def rnd(seed, *shape):
    g = np.random.Generator(np.random.PCG64(seed))
    return ops.bf16_round(g.standard_normal(shape).astype(np.float32))


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().bfloat16()


def bounds(q, k, v, out, mags, scale):
    """|error| per element. Logits: d exact products summed in fp32 (truncated
    at worst) and scaled: e = (2 d + 16) 2^-24 scale sum |q| |k|, plus exp2's
    2^-22 and its argument's 2^-23 of at most 128; the weights move by 2 e. p is
    rounded to bf16 (2^-8 of each term) in the products but not in their sum,
    the output once more; the running reference may lie 2^8 below the maximum,
    which costs nothing relative."""
    d = q.shape[-1]
    e = (2 * d + 16) * 2.0 ** -24 * scale * np.abs(q).sum(-1, keepdims=True) * np.abs(k).max()
    e = e + 2.0 ** -22 + 128 * 2.0 ** -23
    return 2 * e * mags + 2.0 ** -8 * (mags + np.abs(out)) * 1.02 + 2.0 ** -18 * mags


def call(resa, q, k, v, starts, cap, longest=None, scale=None, out=None, desc=True):
    T, Hq, d = q.shape
    H, B = k.shape[1], len(starts) - 1
    qt, kt, vt = dev(q), dev(k), dev(v)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    kc = torch.full((B, H, cap, d), 5.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 6.0)
    ds = torch.full((B, H, cap // 16, 2, d), 7.0, dtype=torch.bfloat16, device="cuda") if desc else None
    out = torch.full_like(qt, 9.0) if out is None else out
    ws = resa.alloc_workspace(resa.dims_for(kc, Hq), cap)
    longest = longest or max(int(b - a) for a, b in zip(starts[:-1], starts[1:]))
    scale = scale or 1.0 / math.sqrt(d)
    resa.prefill_packed(qt, kt, vt, st, longest, kc, vc, ds, scale, out, ws)
    return out, kc, vc, ds, ws, scale


def check(resa, q, k, v, starts, got, kc, vc, ds, scale, rows=None):
    G = q.shape[1] // k.shape[1]
    o = got.double().cpu().numpy()
    kcn, vcn = kc.float().cpu().numpy(), vc.float().cpu().numpy()
    dn = None if ds is None else ds.float().cpu().numpy()
    inside = np.zeros(q.shape[0], bool)
    for b, (a, e) in enumerate(zip(starts[:-1], starts[1:])):
        n = e - a
        inside[a:e] = True
        for h in range(k.shape[1]):
            assert np.array_equal(kcn[b, h, :n], k[a:e, h]) and (kcn[b, h, n:] == 5.0).all()
            assert np.array_equal(vcn[b, h, :n], v[a:e, h]) and (vcn[b, h, n:] == 6.0).all()
            if dn is not None:
                nb = (n + 15) // 16
                assert np.array_equal(dn[b, h, :nb], ops.descriptors(k[a:e, h], n))
                assert (dn[b, h, nb:] == 7.0).all()
        if n == 0:
            continue
        at = np.arange(n) if rows is None or n <= rows else np.unique(
            np.concatenate([np.arange(40), np.linspace(0, n - 1, rows).astype(int), np.arange(n - 40, n)]))
        for h in range(q.shape[1]):
            kk, vv = k[a:e, h // G].astype(np.float64), v[a:e, h // G].astype(np.float64)
            qq = q[a:e, h][at].astype(np.float64)
            z = np.where(np.arange(n)[None] <= at[:, None], qq @ kk.T * scale, -np.inf)
            p = np.exp(z - z.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            ref, mags = p @ vv, p @ np.abs(vv)
            err = np.abs(o[a:e, h][at] - ref)
            bo = bounds(qq, kk, vv, ref, mags, scale)
            assert (err <= bo).all(), (b, h, float((err / bo).max()))
    assert (o[~inside] == 9.0).all(), "rows of no sequence were written"


def starts_of(lens, lead=0):
    return [lead + int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 8])
@pytest.mark.parametrize("lens", [[1], [128], [1, 0, 31, 33, 200], [63, 64, 65, 127, 129], [300, 257]])
@pytest.mark.parametrize("longest", [None, 2100])       # (one tile per CTA, two)
def test_packed(resa, d, G, lens, longest):
    H, st = 2, starts_of(lens)
    q, k, v = rnd(1, st[-1], H * G, d), rnd(2, st[-1], H, d), rnd(3, st[-1], H, d)
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, st, 320 if longest is None else 2112, longest)
    assert resa.workspace_status(ws) == resa.RESA_OK
    check(resa, q, k, v, st, out, kc, vc, ds, scale)


def test_rows_before_and_behind_the_sequences_stay(resa):
    lens = [40, 1, 150]
    st = starts_of(lens, lead=7)
    T = st[-1] + 13
    q, k, v = rnd(1, T, 8, 128), rnd(2, T, 2, 128), rnd(3, T, 2, 128)
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, st, 160, longest=160)
    check(resa, q, k, v, st, out, kc, vc, ds, scale)
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, st, 160, desc=False)
    check(resa, q, k, v, st, out, kc, vc, ds, scale)
    assert resa.workspace_status(ws) == resa.RESA_OK


@pytest.mark.parametrize("short", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_of_a_neighbour_do_not_leak(resa, bad, short):
    """Keys, values and queries of one sequence that are not finite change no
    bit of another's outputs, though their key tiles hold rows of both."""
    lens = [50, 77, 30, 129]
    st = starts_of(lens)
    q, k, v = rnd(1, st[-1], 8, 64), rnd(2, st[-1], 2, 64), rnd(3, st[-1], 2, 64)
    cap, longest = (144, None) if short else (2112, 2100)
    clean = call(resa, q, k, v, st, cap, longest)[0]
    q2, k2, v2 = q.copy(), k.copy(), v.copy()
    for x in (q2, k2, v2):
        x[st[1]:st[2]] = bad
        x[st[3] + 128:] = bad                       # behind the last sequence's first tile
    out = call(resa, q2, k2, v2, st, cap, longest)[0]
    for i in (0, 2):
        assert torch.equal(out[st[i]:st[i + 1]], clean[st[i]:st[i + 1]])
    assert torch.equal(out[st[3]:st[3] + 128], clean[st[3]:st[3] + 128])


@pytest.mark.parametrize("longest", [None, 2100])
def test_large_logits(resa, longest):
    """Logits of some hundreds: maxima that grow along the row (rescaling), and
    weights that vanish."""
    n = 700
    q, k, v = rnd(1, n, 4, 128), rnd(2, n, 1, 128), rnd(3, n, 1, 128)
    k *= np.linspace(0.1, 16, n).astype(np.float32)[:, None, None]
    k = ops.bf16_round(k)
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, [0, n], 2112, longest, scale=1.0)
    o = out.double().cpu().numpy()
    for h in range(4):
        z = q[:, h].astype(np.float64) @ k[:, 0].astype(np.float64).T
        z = np.where(np.tril(np.ones((n, n), bool)), z, -np.inf)
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        ref, mags = p @ v[:, 0], p @ np.abs(v[:, 0]).astype(np.float64)
        # |logit| up to 1500 in log2 units: the argument's rounding is 1500 2^-23,
        # and the product of two roundings of the logit's sum
        e = (2 * 128 + 16) * 2.0 ** -24 * np.abs(q[:, h]).sum(-1, keepdims=True) * np.abs(k).max() + 3000 * 2.0 ** -23
        assert (np.abs(o[:, h] - ref) <= 2 * e * mags + 2.0 ** -8 * (mags + np.abs(ref)) * 1.02).all()
    assert resa.workspace_status(ws) == resa.RESA_OK


def test_many_sequences(resa):
    g = np.random.default_rng(0)
    lens = g.integers(0, 20, 333).tolist()
    st = starts_of(lens)
    q, k, v = rnd(1, st[-1], 4, 64), rnd(2, st[-1], 1, 64), rnd(3, st[-1], 1, 64)
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, st, 32)
    assert resa.workspace_status(ws) == resa.RESA_OK
    check(resa, q, k, v, st, out, kc, vc, ds, scale)


@pytest.mark.parametrize("d,H,G", [(128, 2, 4), (64, 1, 8), (128, 1, 1), (128, 2, 3)])
def test_long_sequences(resa, d, H, G):
    lens = [2500, 4099, 1]
    st = starts_of(lens)
    q, k, v = rnd(1, st[-1], H * G, d), rnd(2, st[-1], H, d), rnd(3, st[-1], H, d)
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, st, 4112)
    assert resa.workspace_status(ws) == resa.RESA_OK
    check(resa, q, k, v, st, out, kc, vc, ds, scale, rows=200)
    again = call(resa, q, k, v, st, 4112)[0]
    assert torch.equal(out, again)


def test_agrees_with_the_fixed_length_prefill(resa):
    """Equal lengths: the packed call and resa_prefill compute the same thing
    (in another tiling, so to rounding) and leave the same descriptors."""
    B, n, H, G, d = 2, 500, 2, 4, 128
    q, k, v = rnd(1, B * n, H * G, d), rnd(2, B * n, H, d), rnd(3, B * n, H, d)
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, [0, n, 2 * n], 512)
    o2 = torch.zeros(B, n, H * G, d, dtype=torch.bfloat16, device="cuda")
    d2 = torch.full_like(ds, 7.0)
    resa.prefill(dev(q).view(B, n, H * G, d), kc, vc, d2, n, scale, o2, ws)
    assert torch.equal(ds, d2)
    diff = (out.view_as(o2).float() - o2.float()).abs()
    assert (diff <= 4 * 2.0 ** -8 * (o2.float().abs() + 1.0)).all()


def test_bad_starts_are_cut_and_flagged(resa):
    T = 200
    q, k, v = rnd(1, T, 4, 64), rnd(2, T, 1, 64), rnd(3, T, 1, 64)
    for starts, eff in (([0, 50, 40, 200], [(0, 50), (50, 50), (40, 200)]),
                        ([-5, 60, 1000, 1000], [(0, 60), (60, 200), (200, 200)])):
        out, kc, vc, ds, ws, scale = call(resa, q, k, v, starts, 208, longest=200)
        assert resa.workspace_status(ws) == resa.RESA_ERR_BAD_INDEX
        o = out.double().cpu().numpy()
        a, e = eff[0]
        ref = ops.packed_causal(q[a:e], k[a:e], v[a:e], [0, e - a], scale)
        assert np.abs(o[a:e] - ref).max() < 0.05
    # a sequence longer than `longest`: its first `longest` tokens
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, [0, 150, 200], 208, longest=60)
    assert resa.workspace_status(ws) == resa.RESA_ERR_BAD_INDEX
    o = out.double().cpu().numpy()
    assert np.abs(o[:60] - ops.packed_causal(q[:60], k[:60], v[:60], [0, 60], scale)).max() < 0.05
    assert (o[60:150] == 9.0).all() and (kc[0, :, 60:] == 5.0).all()


def test_prefill_then_decode_ragged(resa):
    """As used: packed prompts, then sparse steps on the ragged batch (all
    blocks kept), and a graph of the prefill replayed on other lengths."""
    H, G, d, cap, B = 2, 4, 128, 272, 3
    lens = [100, 17, 250]
    st = starts_of(lens)
    T = 400
    q, k, v = rnd(1, T, H * G, d), rnd(2, T, H, d), rnd(3, T, H, d)
    qt, kt, vt = dev(q), dev(k), dev(v)
    kc = torch.zeros(B, H, cap, d, dtype=torch.bfloat16, device="cuda")
    vc, ds = torch.zeros_like(kc), torch.zeros(B, H, cap // 16, 2, d, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(qt)
    ws = resa.alloc_workspace(resa.dims_for(kc, H * G), cap)
    stt = torch.tensor([0, 0, 0, 0], dtype=torch.int32, device="cuda")
    scale = 1.0 / math.sqrt(d)
    resa.prefill_packed(qt, kt, vt, stt, 260, kc, vc, ds, scale, out, ws)   # nothing to do
    torch.cuda.synchronize()
    assert not out.any() and not kc.any()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        resa.prefill_packed(qt, kt, vt, stt, 260, kc, vc, ds, scale, out, ws)
    stt.copy_(torch.tensor(st, dtype=torch.int32))
    g.replay()
    dq, dk, dv = (rnd(50 + i, B, x, d) for i, x in enumerate((H * G, H, H)))
    lt = torch.tensor([x + 1 for x in lens], dtype=torch.int32, device="cuda")
    o1 = torch.zeros(B, H * G, d, dtype=torch.bfloat16, device="cuda")
    resa.decode_sparse_varlen(dev(dq), dev(dk), dev(dv), kc, vc, ds, lt, max(lens) + 1, 1.0, 1, scale, o1, ws)
    assert resa.workspace_status(ws) == resa.RESA_OK
    o = o1.double().cpu().numpy()
    for b in range(B):
        for h in range(H):
            kk = np.concatenate([k[st[b]:st[b + 1], h], dk[b, h][None]])
            vv = np.concatenate([v[st[b]:st[b + 1], h], dv[b, h][None]])
            ref, _, p = ops.attend_row(dq[b, h * G:(h + 1) * G], kk, vv, scale)
            tol = 2.0 ** -8 * (p @ np.abs(vv) + np.abs(ref)) * 1.02 + 1e-5
            assert (np.abs(o[b, h * G:(h + 1) * G] - ref) <= tol).all()


@pytest.mark.parametrize("longest", [None, 2100])
@pytest.mark.parametrize("size", [3e4, 1e5, 1e6])
def test_large_finite_logits(resa, longest, size):
    """Queries and keys of 1e4 to 1e6, as the header allows: logits of 2^30 and
    more in log2 units, whose rounding is wider than any weight's exponent.
    Where a row's largest is ahead of the next by more than both may be off, the
    definition gives its value alone."""
    lens, G, d = [300, 77], 4, 128
    st, scale = starts_of(lens), 1.0 / math.sqrt(d)
    q, k, v = rnd(1, st[-1], G, d), rnd(2, st[-1], 1, d), rnd(3, st[-1], 1, d)
    q, k = ops.bf16_round(q * np.float32(size)), ops.bf16_round(k * np.float32(size))
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, st, 2112, longest, scale=scale)
    assert resa.workspace_status(ws) == resa.RESA_OK
    o = out.double().cpu().numpy()
    assert np.isfinite(o).all()
    clear = 0
    for a, b in zip(st[:-1], st[1:]):
        n = b - a
        for h in range(G):
            qq, kk = q[a:b, h].astype(np.float64), k[a:b, 0].astype(np.float64)
            z = np.where(np.tril(np.ones((n, n), bool)), qq @ kk.T * scale, -np.inf)
            # (as in `bounds`, and the rounding to log2 units)
            e = (2 * d + 16) * 2.0 ** -24 * scale * np.abs(qq).sum(-1) * np.abs(kk).max()
            e = e + 2.0 ** -22 * np.abs(z[np.isfinite(z)]).max()
            top = np.sort(z, -1)[:, -2:]
            gap = np.full(n, np.inf)
            gap[1:] = top[1:, 1] - top[1:, 0]
            for i in np.flatnonzero(gap > 2 * e + 100):
                clear += 1
                want = v[a + z[i].argmax(), 0].astype(np.float64)
                assert (np.abs(o[a + i, h] - want) <= 2.0 ** -8 * 2.02 * np.abs(want)).all(), (a + i, h)
    assert clear > st[-1] * G // 2


@pytest.mark.parametrize("longest", [None, 2100])
def test_equal_logits_of_any_size(resa, longest):
    """Heads whose logits are all equal, +-2^20 to 2^40 in log2 units: the running mean."""
    n, G, d = 140, 8, 64
    q, k, v = np.zeros((n, G, d), np.float32), np.zeros((n, 1, d), np.float32), rnd(3, n, 1, d)
    q[:, :, 0] = ops.bf16_round((2.0 ** np.linspace(10, 30, G) * np.array([1, -1] * (G // 2))).astype(np.float32))
    k[:, :, 0] = 1024.0
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, [0, n], 2112, longest, scale=1.0)
    o = out.double().cpu().numpy()
    want = np.cumsum(v[:, 0].astype(np.float64), 0) / np.arange(1, n + 1)[:, None]
    # weights of one size each, so that their rounding to bf16 is one factor of
    # all of them (up to 2^-8); sums of n terms; the output's rounding
    tol = 2.0 ** -8 * 2.02 * np.abs(want) + n * 2.0 ** -23 * np.abs(v).max()
    for h in range(G):
        assert (np.abs(o[:, h] - want) <= tol).all(), h


@pytest.mark.parametrize("longest", [None, 2100])
@pytest.mark.parametrize("desc", [True, False])
def test_without_caches(resa, longest, desc):
    """Caches left out: the same outputs and descriptors, bit for bit."""
    lens, H, G, d = [200, 0, 77, 16], 2, 4, 128
    st = starts_of(lens)
    q, k, v = rnd(1, st[-1], H * G, d), rnd(2, st[-1], H, d), rnd(3, st[-1], H, d)
    cap = 208 if longest is None else 2112
    want, kc, _, ds, ws, scale = call(resa, q, k, v, st, cap, longest)
    out, d2 = torch.full_like(want, 9.0), torch.full_like(ds, 7.0) if desc else None
    resa.prefill_packed(dev(q), dev(k), dev(v), torch.tensor(st, dtype=torch.int32, device="cuda"),
                        longest or max(lens), None, None, d2, scale, out, ws)
    assert resa.workspace_status(ws) == resa.RESA_OK
    assert torch.equal(out, want) and (d2 is None or torch.equal(d2, ds))
    # and a bound that the descriptors have no room for is refused
    if desc:
        with pytest.raises(resa.ResaError) as e:
            resa.prefill_packed(dev(q), dev(k), dev(v), torch.tensor(st, dtype=torch.int32, device="cuda"),
                                cap + 1, None, None, d2, scale, out, ws)
        assert e.value.status == resa.RESA_ERR_CAPACITY


@pytest.mark.parametrize("T", [2000, 2300])              # (one tile per CTA, two)
@pytest.mark.parametrize("starts,eff", [([0, 1500, 700, 1900], {0: (0, 1500)}),
                                        ([5, 3, 900, 10, 4, 1300, 0], {}), ([2000, 0, 100], {}),
                                        ([0, 40, 30, 60, 100, 2000], {0: (0, 40), 3: (60, 100), 4: (100, 2000)})])
def test_starts_out_of_order_share_no_token(resa, starts, eff, T):
    """A sequence that begins below an earlier start is left out, so every row
    is the one sequence's it belongs to, whichever CTA comes last."""
    H, G, d = 1, 4, 64
    q, k, v = rnd(1, T, H * G, d), rnd(2, T, H, d), rnd(3, T, H, d)
    out, kc, vc, ds, ws, scale = call(resa, q, k, v, starts, 2304, T)
    assert resa.workspace_status(ws) == resa.RESA_ERR_BAD_INDEX
    o, inside = out.double().cpu().numpy(), np.zeros(T, bool)
    for b in range(len(starts) - 1):
        a, e = eff.get(b, (0, 0))
        inside[a:e] = True
        kn = kc[b, 0].float().cpu().numpy()
        assert np.array_equal(kn[:e - a], k[a:e, 0]) and (kn[e - a:] == 5.0).all()
        assert (ds[b, 0, (e - a + 15) // 16:] == 7.0).all()
        if e > a:
            ref = ops.packed_causal(q[a:e], k[a:e], v[a:e], [0, e - a], scale)
            mags = ops.packed_causal(q[a:e], k[a:e], np.abs(v[a:e]), [0, e - a], scale)
            for h in range(H * G):
                bo = bounds(q[a:e, h].astype(np.float64), k[a:e, 0], v[a:e, 0], ref[:, h], mags[:, h], scale)
                assert (np.abs(o[a:e, h] - ref[:, h]) <= bo).all()
    assert (o[~inside] == 9.0).all()
