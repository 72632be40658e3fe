"""Attention weights and eviction on the GPU against their plain definitions
(oracle/cache_ops.py)."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as ops

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def resa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_quest_b200 as m
    return m


def rnd(seed, *shape, dtype="bf16"):
    x = np.random.Generator(np.random.PCG64(seed)).standard_normal(shape).astype(np.float32)
    return ops.bf16_round(x) if dtype == "bf16" else x


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(DT[dtype])


# ---------------------------------------------------------------------- weights

def weight_bounds(q, k, w, scale):
    """Bound on the relative error of one head's weights: a logit's (sums of d
    exact or once-rounded products in fp32, truncated at worst) enters twice,
    itself and through the normaliser; exp2 and its argument (below 128 in
    magnitude) add the rest."""
    d = q.shape[-1]
    e = (2 * d + 16) * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q)).max() + 2.0 ** -22 + 128 * 2.0 ** -23
    return 2 * e + 2.0 ** -20


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 3), (128, 4), (128, 8)])
@pytest.mark.parametrize("lens,ragged", [([1, 1], False), ([17, 17], False), ([2100, 2100], False),
                                         ([1, 900, 33, 16], True)])
def test_weights_of_a_step(resa, dtype, d, G, lens, ragged):
    B, H, cap, n = len(lens), 2, 2128, max(lens)
    k, v = rnd(1, B, H, cap, d, dtype=dtype), rnd(2, B, H, cap, d, dtype=dtype)
    q, kn, vn = (rnd(3 + i, B, x, d, dtype=dtype) for i, x in enumerate((H * G, H, H)))
    for b, x in enumerate(lens):
        k[b, :, x:], v[b, :, x:] = np.nan, np.nan
    kt, vt = dev(k, dtype), dev(v, dtype)
    desc = torch.zeros(B, H, cap // 16, 2, d, dtype=DT[dtype], device="cuda")
    w0 = np.random.default_rng(9).random((B, H, cap)).astype(np.float32)
    for b, x in enumerate(lens):
        w0[b, :, x - 1] = np.nan           # the appended token's slot: whatever it held
        w0[b, :, x:] = -5.0
    wt = torch.from_numpy(w0).cuda()
    qt, knt, vnt = dev(q, dtype), dev(kn, dtype), dev(vn, dtype)
    dims = resa.dims_for(kt, H * G)
    ws = resa.alloc_weights_workspace(dims, n)
    out, lse = torch.empty_like(qt), torch.empty(B, H * G, device="cuda")
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda") if ragged else None
    scale = 1.0 / math.sqrt(d)
    k2, v2, d2 = kt.clone(), vt.clone(), desc.clone()
    resa.decode_dense_weights(qt, knt, vnt, kt, vt, desc, wt, n, scale, out, lse, ws, lens=lt)
    assert resa.workspace_status(ws) == resa.RESA_OK
    # the same outputs, cache and descriptors as the plain dense step
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws2 = resa.alloc_workspace(dims, n)
    if ragged:
        resa.decode_dense_varlen(qt, knt, vnt, k2, v2, d2, lt, n, scale, o2, ws2, lse=l2)
    else:
        resa.decode_dense(qt, knt, vnt, k2, v2, d2, n, scale, o2, ws2, lse=l2)
    assert torch.equal(kt.nan_to_num(), k2.nan_to_num()) and torch.equal(vt.nan_to_num(), v2.nan_to_num())
    assert torch.equal(desc, d2)
    got = wt.cpu().numpy()
    kf, vf = k2.double().cpu().numpy(), v2.double().cpu().numpy()
    if dtype == "bf16":
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    else:
        # (a kernel of its own in fp32) sums of d products and of n weighted
        # values, each term rounded once: n 2^-24 of the magnitudes at worst
        on, ln = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, x in enumerate(lens):
            for h in range(H):
                qs = q[b, h * G:(h + 1) * G].astype(np.float64)
                o, e, w = ops.attend_row(qs, kf[b, h, :x], vf[b, h, :x], scale)
                for i in range(G):
                    rel = weight_bounds(qs[i], kf[b, h, :x], w[i], scale)
                    mags = w[i] @ np.abs(vf[b, h, :x])
                    assert (np.abs(on[b, h * G + i] - o[i]) <= (rel + (x + 64) * 2.0 ** -24) * mags + 1e-37).all()
                    assert abs(ln[b, h * G + i] - e[i]) <= rel + (x + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(e[i])

    def one_step(prev, fresh):
        want, tol = prev.astype(np.float64), np.zeros(prev.shape)
        for b, x in enumerate(lens):
            for h in range(H):
                qs = q[b, h * G:(h + 1) * G].astype(np.float64)
                _, _, w = ops.attend_row(qs, kf[b, h, :x], vf[b, h, :x], scale)
                rel = max(weight_bounds(qs[i], kf[b, h, :x], w[i], scale) for i in range(G))
                if fresh:
                    want[b, h, x - 1] = 0.0
                want[b, h, :x] += w.sum(0)
                tol[b, h, :x] = rel * w.sum(0) + 2.0 ** -23 * np.abs(want[b, h, :x]) + 1e-37
        return want, tol

    want, tol = one_step(w0, True)
    assert (np.abs(got - want) <= tol).all()
    # a second pass without a new token adds to every slot, the newest too
    resa.decode_dense_weights(qt, None, None, kt, vt, None, wt, n, scale, out, None, ws, lens=lt)
    assert resa.workspace_status(ws) == resa.RESA_OK
    want, tol = one_step(got, False)
    assert (np.abs(wt.cpu().numpy() - want) <= tol).all()
    assert dtype == "f32" or torch.equal(out, o2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_below_the_fp32_range_weigh_nothing(resa, dtype):
    # tokens 0 .. 31 (the first blocks of two warps): logits near -1e39; the
    # others' keys leave channel 0 out
    B, H, G, d, n, scale = 1, 2, 4, 128, 64, 1.0 / math.sqrt(128)
    k, v = rnd(1, B, H, n, d, dtype=dtype), rnd(2, B, H, n, d, dtype=dtype)
    q = rnd(3, B, H * G, d, dtype=dtype)
    k[..., 0] = 0.0
    k[:, :, :32, 0], q[:, :, 0] = ops.bf16_round(np.float32(-1e22)), ops.bf16_round(np.float32(1e18))
    kt, vt, qt = dev(k, dtype), dev(v, dtype), dev(q, dtype)
    wt = torch.zeros(B, H, n, device="cuda")
    out, lse = torch.empty_like(qt), torch.empty(B, H * G, device="cuda")
    ws = resa.alloc_weights_workspace(resa.dims_for(kt, H * G), n)
    resa.decode_dense_weights(qt, None, None, kt, vt, None, wt, n, scale, out, lse, ws)
    assert resa.workspace_status(ws) == resa.RESA_OK
    got, on = wt.double().cpu().numpy(), out.double().cpu().numpy()
    q[:, :, 0] = 0.0
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24   # a rounding of a weight, of an output
    for h in range(H):
        qs = q[0, h * G:(h + 1) * G].astype(np.float64)
        kf, vf = k[0, h, 32:].astype(np.float64), v[0, h, 32:].astype(np.float64)
        o, _, w = ops.attend_row(qs, kf, vf, scale)
        rel = max(weight_bounds(qs[i], kf, w[i], scale) for i in range(G))
        assert (got[0, h, :32] == 0).all()
        assert (np.abs(got[0, h, 32:] - w.sum(0)) <= rel * w.sum(0) + 1e-37).all()
        tol = (rel + 1.01 * half + 96 * 2.0 ** -24) * (w @ np.abs(vf)) + half * np.abs(o)
        assert (np.abs(on[0, h * G:(h + 1) * G] - o) <= tol).all()


# --------------------------------------------------------------------- eviction

def run_evict(resa, k, v, w, lens, budget, recent, dtype, cap_out, bound=None, sentinel=3.0):
    B, H, cap, d = k.shape
    kt, vt, wt = dev(k, dtype), dev(v, dtype), torch.from_numpy(w).cuda()
    ko = torch.full((B, H, cap_out, d), sentinel, dtype=DT[dtype], device="cuda")
    vo = torch.full_like(ko, sentinel)
    do = torch.full((B, H, cap_out // 16, 2, d), sentinel, dtype=DT[dtype], device="cuda")
    wo = torch.full((B, H, cap_out), sentinel, device="cuda")
    kept = torch.full((B, H, budget), -7, dtype=torch.int32, device="cuda")
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda") if bound or len(set(lens)) > 1 else None
    n = bound or max(lens)
    ws = resa.alloc_workspace(resa.dims_for(kt, H), n)
    resa.evict(kt, vt, wt, n, budget, recent, ko, vo, do, wo, kept, H, ws, lens=lt)
    assert resa.workspace_status(ws) == resa.RESA_OK
    got = [x.float().cpu().numpy() for x in (ko, vo, do, wo)] + [kept.cpu().numpy()]
    for b in range(B):
        for h in range(H):
            idx = ops.evict_row(w[b, h], lens[b], budget, recent)
            m, nb = len(idx), (len(idx) + 15) // 16
            assert np.array_equal(got[4][b, h, :m], idx), (b, h)
            assert (got[4][b, h, m:] == -1).all()
            assert np.array_equal(got[0][b, h, :m], k[b, h, idx]) and (got[0][b, h, m:] == sentinel).all()
            assert np.array_equal(got[1][b, h, :m], v[b, h, idx]) and (got[1][b, h, m:] == sentinel).all()
            assert np.array_equal(got[3][b, h, :m], w[b, h, idx], equal_nan=True)
            assert (got[3][b, h, m:] == sentinel).all()
            assert np.array_equal(got[2][b, h, :nb], ops.descriptors(k[b, h, idx], m))
            assert (got[2][b, h, nb:] == sentinel).all()
    return got


def weights_of(kind, B, H, cap, seed=4):
    g = np.random.default_rng(seed)
    if kind == "heavy":
        return np.exp(2.5 * g.standard_normal((B, H, cap))).astype(np.float32)
    if kind == "equal":
        return np.full((B, H, cap), 0.25, np.float32)
    if kind == "few":                       # long runs of ties around the threshold
        return g.integers(0, 3, (B, H, cap)).astype(np.float32)
    w = g.standard_normal((B, H, cap)).astype(np.float32)
    w.ravel()[::7], w.ravel()[3::11], w.ravel()[5::13] = np.nan, -0.0, 0.0
    w.ravel()[::17], w.ravel()[1::19] = np.inf, -np.inf
    w.ravel()[2::23] = 1e-42                # subnormal
    return w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["heavy", "equal", "few", "odd"])
@pytest.mark.parametrize("n,budget,recent", [(2, 1, 0), (2, 1, 1), (33, 17, 5), (1000, 999, 1),
                                             (1000, 16, 16), (5003, 1200, 64), (777, 777, 5)])
def test_evict(resa, dtype, d, kind, n, budget, recent):
    B, H, cap = 1, 2, (n + 15) // 16 * 16
    k, v = rnd(1, B, H, cap, d, dtype=dtype), rnd(2, B, H, cap, d, dtype=dtype)
    run_evict(resa, k, v, weights_of(kind, B, H, cap), [n], budget, recent, dtype,
              (budget + 15) // 16 * 16 + 16)


@pytest.mark.parametrize("kind", ["heavy", "few", "odd"])
def test_evict_ragged(resa, kind):
    """Rows above, at and below the budget."""
    lens = [3000, 1, 512, 513, 40]
    B, H, cap, d = len(lens), 2, 3008, 64
    k, v = rnd(1, B, H, cap, d), rnd(2, B, H, cap, d)
    run_evict(resa, k, v, weights_of(kind, B, H, cap), lens, 512, 33, "bf16", 528)
    run_evict(resa, k, v, weights_of(kind, B, H, cap), lens, 512, 33, "bf16", 528, bound=3008)


def test_evict_budget_above_every_length(resa):
    k, v = rnd(1, 1, 2, 64, 64), rnd(2, 1, 2, 64, 64)
    run_evict(resa, k, v, weights_of("heavy", 1, 2, 64), [50], 100, 10, "bf16", 112)


@pytest.mark.parametrize("n", [8192, 8193, 65537, 131072])
def test_evict_at_the_kernels_bounds(resa, n):
    """Lengths at which the selection changes its number of CTAs or of keys per
    thread."""
    cap = (n + 15) // 16 * 16
    k, v = rnd(1, 1, 1, cap, 64), rnd(2, 1, 1, cap, 64)
    for kind in ("heavy", "equal", "few", "odd"):
        run_evict(resa, k, v, weights_of(kind, 1, 1, cap), [n], n // 3, 17, "bf16", (n // 3 + 15) // 16 * 16)


def test_evict_long_row(resa):
    n = 262144 + 333
    cap = (n + 15) // 16 * 16
    k, v = rnd(1, 1, 1, cap, 64), rnd(2, 1, 1, cap, 64)
    run_evict(resa, k, v, weights_of("heavy", 1, 1, cap), [n], 20000, 128, "bf16", 20000)
    run_evict(resa, k, v, weights_of("few", 1, 1, cap), [n], 200001, 0, "bf16", 200016)


def test_steps_then_eviction_then_steps(resa):
    """The operators as they are used: steps that add up weights, a cut to the
    budget, and sparse and dense steps on what is left."""
    B, H, G, d, n0, steps, budget = 2, 2, 4, 64, 300, 24, 128
    cap, small = 352, 160
    scale = 1.0 / math.sqrt(d)
    k, v = rnd(1, B, H, cap, d), rnd(2, B, H, cap, d)
    kt, vt = dev(k, "bf16"), dev(v, "bf16")
    desc = torch.zeros(B, H, cap // 16, 2, d, dtype=torch.bfloat16, device="cuda")
    resa.build_desc(kt, n0, desc, H * G)
    wt = torch.zeros(B, H, cap, device="cuda")
    ws = resa.alloc_weights_workspace(resa.dims_for(kt, H * G), cap)
    out = torch.empty(B, H * G, d, dtype=torch.bfloat16, device="cuda")
    w = np.zeros((B, H, cap))
    for s in range(steps):
        q, kn, vn = (rnd(100 + 3 * s + i, B, x, d) for i, x in enumerate((H * G, H, H)))
        n = n0 + s + 1
        resa.decode_dense_weights(dev(q, "bf16"), dev(kn, "bf16"), dev(vn, "bf16"), kt, vt, desc, wt, n,
                                  scale, out, None, ws)
        k[:, :, n - 1], v[:, :, n - 1] = kn, vn
        for b in range(B):
            for h in range(H):
                w[b, h, :n] += ops.attend_row(q[b, h * G:(h + 1) * G], k[b, h, :n], v[b, h, :n], scale)[2].sum(0)
    n = n0 + steps
    ko = torch.zeros(B, H, small, d, dtype=torch.bfloat16, device="cuda")
    vo, do = torch.zeros_like(ko), torch.zeros(B, H, small // 16, 2, d, dtype=torch.bfloat16, device="cuda")
    wo = torch.zeros(B, H, small, device="cuda")
    kept = torch.zeros(B, H, budget, dtype=torch.int32, device="cuda")
    resa.evict(kt, vt, wt, n, budget, 32, ko, vo, do, wo, kept, H * G, ws)
    got = kept.cpu().numpy()
    w32 = wt.cpu().numpy()
    # sums agree to fp32 accuracy; the choice is exact on the sums the GPU holds
    assert np.allclose(w32[:, :, :n], w[:, :, :n], rtol=steps * 2.0 ** -15, atol=0)
    for b in range(B):
        for h in range(H):
            assert np.array_equal(got[b, h], ops.evict_row(w32[b, h], n, budget, 32))
    # decoding goes on from the small cache
    q, kn, vn = (rnd(900 + i, B, x, d) for i, x in enumerate((H * G, H, H)))
    ws2 = resa.alloc_workspace(resa.dims_for(ko, H * G), small)
    lse = torch.empty(B, H * G, device="cuda")
    resa.decode_sparse(dev(q, "bf16"), dev(kn, "bf16"), dev(vn, "bf16"), ko, vo, do, budget + 1, 1.0, 1, scale,
                       out, ws2, lse=lse)
    o = out.double().cpu().numpy()
    for b in range(B):
        for h in range(H):
            ks = np.concatenate([k[b, h, got[b, h]], kn[b, h][None]])
            vs = np.concatenate([v[b, h, got[b, h]], vn[b, h][None]])
            ref, _, p = ops.attend_row(q[b, h * G:(h + 1) * G], ks, vs, scale)
            # p and the output are rounded to bf16 (2^-8 each)
            tol = 2.0 ** -8 * (p @ np.abs(vs) + np.abs(ref)) * 1.02 + 1e-5
            assert (np.abs(o[b, h * G:(h + 1) * G] - ref) <= tol).all()
    assert resa.workspace_status(ws) == resa.RESA_OK and resa.workspace_status(ws2) == resa.RESA_OK


def test_captured_step_and_eviction(resa):
    """A step and a cut captured in one graph, replayed on other queries and
    lengths, equal the eager calls bit for bit."""
    B, H, G, d, cap, budget = 2, 2, 2, 128, 1024, 200
    k, v = rnd(1, B, H, cap, d), rnd(2, B, H, cap, d)
    kt, vt = dev(k, "bf16"), dev(v, "bf16")
    q, kn, vn = (dev(rnd(5 + i, B, x, d), "bf16") for i, x in enumerate((H * G, H, H)))
    lens = torch.tensor([1000, 150], dtype=torch.int32, device="cuda")
    dims = resa.dims_for(kt, H * G)

    def call(state):
        kc, vc, w, ws, out, ko, vo, do, wo, kept = state
        resa.decode_dense_weights(q, kn, vn, kc, vc, None, w, cap, 0.09, out, None, ws, lens=lens)
        resa.evict(kc, vc, w, cap, budget, 20, ko, vo, do, wo, kept, H * G, ws, lens=lens)

    def state():
        ko = torch.zeros(B, H, 208, d, dtype=torch.bfloat16, device="cuda")
        return (kt.clone(), vt.clone(), torch.zeros(B, H, cap, device="cuda"),
                resa.alloc_weights_workspace(dims, cap), torch.zeros_like(q), ko, torch.zeros_like(ko),
                torch.zeros(B, H, 13, 2, d, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(B, H, 208, device="cuda"),
                torch.zeros(B, H, budget, dtype=torch.int32, device="cuda"))

    a, e = state(), state()
    call(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(a)
    call(e)
    q.copy_(dev(rnd(50, B, H * G, d), "bf16"))
    lens.copy_(torch.tensor([77, 1024], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    call(e)
    torch.cuda.synchronize()
    for x, y in zip(a[2:3] + a[4:], e[2:3] + e[4:]):
        assert torch.equal(x, y)
    assert resa.workspace_status(a[3]) == resa.RESA_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", ["weights", "dense"])
def test_length_out_of_range_is_clamped_and_flagged(resa, dtype, form):
    """A dense step with row lengths of 0 and beyond the bound does what it does
    at the nearest lengths allowed, and reports them."""
    B, H, G, d, n = 3, 2, 2, 64, 100
    k, v = rnd(1, B, H, 112, d, dtype=dtype), rnd(2, B, H, 112, d, dtype=dtype)
    q, kn, vn = (dev(rnd(3 + i, B, x, d, dtype=dtype), dtype) for i, x in enumerate((H * G, H, H)))
    res = []
    for lens, want in (([0, 50, 101], resa.RESA_ERR_BAD_INDEX), ([1, 50, 100], resa.RESA_OK),
                       ([-7, 50, 100], resa.RESA_ERR_BAD_INDEX)):
        kt, vt = dev(k, dtype), dev(v, dtype)
        desc = torch.zeros(B, H, 7, 2, d, dtype=DT[dtype], device="cuda")
        w, out = torch.ones(B, H, 112, device="cuda"), torch.empty_like(q)
        ws = resa.alloc_weights_workspace(resa.dims_for(kt, H * G), n)
        lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if form == "weights":
            resa.decode_dense_weights(q, kn, vn, kt, vt, desc, w, n, 0.125, out, None, ws, lens=lt)
        else:
            resa.decode_dense_varlen(q, kn, vn, kt, vt, desc, lt, n, 0.125, out, ws)
        assert resa.workspace_status(ws) == want, lens
        res.append((out, kt, vt, desc, w))
    for other in (res[0], res[2]):
        assert all(torch.equal(x, y) for x, y in zip(res[1], other))


def test_the_plain_step_also_weighs_such_logits_with_nothing(resa):
    """The step that keeps weights gives resa_decode_dense's outputs bit for bit,
    also where a warp's first logits all overflow to minus infinity; and so does
    the list of all blocks, in its own cut of the work."""
    B, H, G, d, n, scale = 1, 2, 4, 128, 64, 1.0 / math.sqrt(128)
    k, v, q = rnd(1, B, H, n, d), rnd(2, B, H, n, d), rnd(3, B, H * G, d)
    k[..., 0] = 0.0
    k[:, :, :32, 0], q[:, :, 0] = ops.bf16_round(np.float32(-1e22)), ops.bf16_round(np.float32(1e18))
    kt, vt, qt = dev(k, "bf16"), dev(v, "bf16"), dev(q, "bf16")
    outs = [torch.empty_like(qt) for _ in range(3)]
    lses = [torch.empty(B, H * G, device="cuda") for _ in range(3)]
    ws = resa.alloc_weights_workspace(resa.dims_for(kt, H * G), n)
    resa.decode_dense_weights(qt, None, None, kt, vt, None, torch.zeros(B, H, n, device="cuda"), n, scale, outs[0],
                              lses[0], ws)
    resa.decode_dense(qt, None, None, kt, vt, None, n, scale, outs[1], ws, lse=lses[1])
    sel = torch.arange(n // 16, dtype=torch.int32, device="cuda").expand(B, H, -1).contiguous()
    resa.attend_blocks(qt, kt, vt, n, sel, scale, outs[2], ws, lse=lses[2])
    assert resa.workspace_status(ws) == resa.RESA_OK
    assert torch.equal(outs[0], outs[1]) and torch.equal(lses[0], lses[1])
    assert torch.equal(outs[0], outs[2]) and bool(torch.isfinite(outs[0]).all())


def test_steps_evictions_and_prompts_at_once(resa):
    """Two streams (given explicitly), a workspace each: packed prompts, steps
    that keep weights and evictions of one stream between those of the other
    give bit for bit what they give alone."""
    B, H, G, d, cap, n = 2, 2, 4, 128, 4112, 4100
    k, v = dev(rnd(1, B, H, cap, d), "bf16"), dev(rnd(2, B, H, cap, d), "bf16")
    q, kn, vn = (dev(rnd(3 + i, B, x, d), "bf16") for i, x in enumerate((H * G, H, H)))
    T = 3000
    pq, pk, pv = (dev(rnd(6 + i, T, x, d), "bf16") for i, x in enumerate((H * G, H, H)))
    dims, scale = resa.dims_for(k, H * G), 1.0 / math.sqrt(d)

    class Job:
        def __init__(self, longest):
            self.longest = longest                   # (one query tile per CTA, or two)
            self.k, self.v, self.w = k.clone(), v.clone(), torch.zeros(B, H, cap, device="cuda")
            self.ws = resa.alloc_weights_workspace(dims, cap)
            self.out, self.lse = torch.zeros_like(q), torch.zeros(B, H * G, device="cuda")
            self.ko, self.vo = (torch.zeros(B, H, 512, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.kept = torch.zeros(B, H, 500, dtype=torch.int32, device="cuda")
            self.pout = torch.zeros_like(pq)
            self.pk, self.pv = torch.zeros_like(k), torch.zeros_like(v)
            self.desc = torch.zeros(B, H, cap // 16, 2, d, dtype=torch.bfloat16, device="cuda")
            self.starts = torch.tensor([0, 1100, T], dtype=torch.int32, device="cuda")

        def run(self, stream):
            resa.prefill_packed(pq, pk, pv, self.starts, self.longest, self.pk, self.pv, self.desc, scale, self.pout,
                                self.ws, stream=stream)
            for _ in range(2):
                resa.decode_dense_weights(q, kn, vn, self.k, self.v, None, self.w, n, scale, self.out, self.lse,
                                          self.ws, stream=stream)
            resa.evict(self.k, self.v, self.w, n, 500, 60, self.ko, self.vo, None, None, self.kept, H * G, self.ws,
                       stream=stream)

        def results(self):
            return [self.w, self.out, self.lse, self.ko, self.vo, self.kept, self.pout, self.pk, self.pv, self.desc]

    alone = []
    for longest in (2000, 4096):
        alone.append(Job(longest))
        for _ in range(5):
            alone[-1].run(torch.cuda.current_stream())
        torch.cuda.synchronize()
    jobs, streams = [Job(2000), Job(4096)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for job, st in zip(jobs, streams):
            job.run(st)
    torch.cuda.synchronize()
    for job, one in zip(jobs, alone):
        assert resa.workspace_status(job.ws) == resa.RESA_OK
        for x, y in zip(job.results(), one.results()):
            assert torch.equal(x, y)
