"""The 4-bit cache on the GPU against its plain definition (oracle/cache_ops.py).

Records are compared byte for byte. Attention is compared with 64-bit softmax
over the values the records stand for; the bounds are worked out per element
(see `bounds`), from the roundings the kernel makes.
"""
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


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rnd(seed, *shape, dtype="bf16"):
    g = np.random.Generator(np.random.PCG64(seed))
    x = g.standard_normal(shape).astype(np.float32)
    return ops.bf16_round(x) if dtype == "bf16" else x


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(DT[dtype])


def special_rows(k, v):
    """Values where a code is easy to get wrong: constant groups, grids whose
    quotients are exact halves, tiny and huge ranges, one outlier."""
    n = k.shape[2]
    rows = [np.zeros(64), np.full(64, -2.5), np.arange(64) % 31 * 0.5, np.arange(64) * 2.0 ** -140,
            np.linspace(-1, 1, 64) * 2.0 ** 59, np.eye(64)[5] * 1e4, np.arange(64) % 2 * 2.0 ** -130,
            -np.arange(64) / 4.0]
    for i, r in enumerate(rows):
        if i < n:
            k[:, :, i, :64] = ops.bf16_round(r.astype(np.float32))
            v[:, :, n - 1 - i, -64:] = ops.bf16_round(r.astype(np.float32))


def kv_inputs(seed, B, H, L, d, dtype, special=True):
    k, v = rnd(seed, B, H, L, d, dtype=dtype), rnd(seed + 1, B, H, L, d, dtype=dtype)
    if special:
        special_rows(k, v)
    return k, v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [16], [17, 5, 48], [47, 33]])
def test_quantize_bytes_and_values(resa, dtype, d, lens):
    B, H, L = len(lens), 3, 64
    k, v = kv_inputs(7, B, H, L, d, dtype)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = np.nan, np.inf          # never read
    ref = ops.kv4_pack(np.nan_to_num(k), np.nan_to_num(v, posinf=0.0), lens)
    kt, vt = dev(k, dtype), dev(v, dtype)
    rec = torch.full((B, H, L // 16, ops.kv4_record_bytes(d)), 0xA5, dtype=torch.uint8, device="cuda")
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    resa.kv4_quantize(kt, vt, max(lens), rec, 2 * H, lens=lt if B > 1 else None)
    got = rec.cpu().numpy()
    for b, n in enumerate(lens):
        m = (n + 15) // 16
        assert np.array_equal(got[b, :, :m], ref[b, :, :m]), f"row {b}"
        assert (got[b, :, m:] == 0xA5).all(), f"row {b}: later records were written"
    # and back: zero + scale * code, rounded once to the type
    kb, vb = torch.full_like(kt, 3.0), torch.full_like(vt, 3.0)
    resa.kv4_dequantize(rec, max(lens), kb, vb, 2 * H, lens=lt if B > 1 else None)
    (kc, ks, kz), (vc, vs, vz) = ops.kv4_unpack(ref, d)
    for got_t, val in ((kb, ops.kv4_value(kc, ks, kz)), (vb, ops.kv4_value(vc, vs, vz))):
        x = got_t.float().cpu().numpy()
        want = val.astype(np.float32)
        want = ops.bf16_round(want) if dtype == "bf16" else want
        for b, n in enumerate(lens):
            assert np.array_equal(x[b, :, :n], want[b, :, :n])
            assert (x[b, :, n:] == 3.0).all()


def test_caches_that_are_only_16_byte_aligned(resa):
    k, v = kv_inputs(3, 1, 2, 48, 64, "bf16")
    rec = torch.zeros(1, 2, 3, ops.kv4_record_bytes(64), dtype=torch.uint8, device="cuda")
    buf = torch.zeros(4, k.size + 8, dtype=torch.bfloat16, device="cuda")
    kt, vt, kb, vb = (b[8:8 + k.size].view(k.shape) for b in buf)
    kt.copy_(dev(k, "bf16")), vt.copy_(dev(v, "bf16"))
    assert kt.data_ptr() % 32 == 16 or vt.data_ptr() % 32 == 16
    resa.kv4_quantize(kt, vt, 48, rec, 2)
    resa.kv4_dequantize(rec, 48, kb, vb, 2)
    for got, (c, s, z) in zip((kb, vb), ops.kv4_unpack(rec.cpu().numpy(), 64)):
        want = ops.bf16_round(ops.kv4_value(c, s, z).astype(np.float32))
        assert np.array_equal(got.float().cpu().numpy(), want)
    assert np.array_equal(rec.cpu().numpy(), ops.kv4_pack(k, v, [48]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_appended_tokens_equal_a_whole_quantisation(resa, dtype, d):
    """35 tokens appended one at a time over stale bytes leave the records (and
    the descriptors) that quantising (and describing) the rows whole does."""
    B, H, G, L, n = 2, 2, 2, 48, 35
    k, v = kv_inputs(11, B, H, L, d, dtype)
    rec = torch.full((B, H, L // 16, ops.kv4_record_bytes(d)), 0xC3, dtype=torch.uint8, device="cuda")
    desc = torch.full((B, H, L // 16, 2, d), 9.0, dtype=DT[dtype], device="cuda")
    q = dev(rnd(3, B, H * G, d, dtype=dtype), dtype)
    out = torch.empty_like(q)
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, q), L)
    kt, vt = dev(k, dtype), dev(v, dtype)
    for t in range(n):
        resa.decode_dense_kv4(q, kt[:, :, t].contiguous(), vt[:, :, t].contiguous(), rec, desc, t + 1,
                              1e-30, out, ws)
    want = ops.kv4_pack(k, v, [n] * B)
    got = rec.cpu().numpy()
    assert np.array_equal(got[:, :, :2], want[:, :, :2])
    # of the open block: the codes and scales of its valid tokens
    (kc, ks, kz), (vc, vs, vz) = ops.kv4_unpack(got, d)
    (rc, rs, rz), (wc, w_s, wz) = ops.kv4_unpack(want, d)
    for a, b in ((kc, rc), (ks, rs), (kz, rz), (vc, wc), (vs, w_s), (vz, wz)):
        assert np.array_equal(a[:, :, :n], b[:, :, :n])
    whole = torch.full_like(desc, 9.0)
    resa.build_desc(kt, n, whole, H * G)
    assert torch.equal(desc, whole)
    assert resa.workspace_status(ws) == resa.RESA_OK


def bounds(q, kc, ks, kz, vc, vs, vz, w, scale, dtype, out):
    """Bounds on one head's |output error| [d] and |log-sum-exp error|.

    Logits: sums over d products (codes and bf16 parts of q are exact; fp32 q
    in three parts loses 2^-24 of it). Any order of fp32 additions of n terms
    errs by at most n 2^-24 times the sum of magnitudes; the tensor cores may
    truncate, which doubles it, and the scale, zero and softmax-scale products
    add a few roundings: e = (2 d + 16) 2^-24 scale sum_c |q_c| (|z| + 15 s)
    with the largest group scale. A logit error e moves weights by 2 e (and
    exp2's own 2^-22 and the 64-bit difference of its argument, |arg| 2^-23
    with |arg| < 128, are added to e).
    Outputs: the weights' error times the largest |v|; in bf16 each p * scale
    is rounded (2^-8 relative to its code part) and so is the output; fp32
    keeps 2^-23 of both; sums of n tokens err by n 2^-23 relative to the sum of
    magnitudes at worst, by sqrt(n)-like amounts in fact: n is small here."""
    d, n = q.shape[-1], w.shape[-1]
    mag = (np.abs(kz) + 15 * ks).max(-1).max()
    e = (2 * d + 16) * 2.0 ** -24 * scale * np.abs(q).sum() * mag + 2.0 ** -22 + 128 * 2.0 ** -23
    part = (vs[..., None] * vc.reshape(n, -1, 64)).reshape(n, d).astype(np.float64)
    codes = w @ part
    mags = w @ (part + np.repeat(np.abs(vz), 64, -1))
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    acc = 2.0 ** -23 * min(n, 4096) + 2.0 ** -20
    return 2 * e * mags + step * (codes + np.abs(out)) * 1.01 + acc * mags, e + acc + 2.0 ** -22 * 64


def check(resa, q, rec, lens, sel, got, lse, scale, dtype, d, H):
    G = q.shape[1] // H
    for b in range(q.shape[0]):
        for g in range(H):
            recs = rec[b, g]
            pos = np.arange(recs.shape[0] * 16)
            if sel is not None:
                recs = recs[sel[b, g]]
                pos = (sel[b, g][:, None] * 16 + np.arange(16)).ravel()
            keep = pos < lens[b]
            (kc, ks, kz), (vc, vs, vz) = [tuple(x[keep] for x in y) for y in ops.kv4_unpack(recs, d)]
            kv, vv = ops.kv4_value(kc, ks, kz), ops.kv4_value(vc, vs, vz)
            o, e, w = ops.attend_row(q[b, g * G:(g + 1) * G], kv, vv, scale)
            for h in range(G):
                bo, be = bounds(q[b, g * G + h], kc, ks, kz, vc, vs, vz, w[h], scale, dtype, o[h])
                err = np.abs(got[b, g * G + h] - o[h])
                assert (err <= bo).all(), (b, g, h, float((err / bo).max()))
                assert abs(lse[b, g * G + h] - e[h]) <= be * (1 + abs(e[h])), (b, g, h)


def run_dense(resa, B, H, G, d, dtype, lens, cap, seed=5, bound=None, stale=True):
    k, v = kv_inputs(seed, B, H, cap, d, dtype, special=False)
    q = rnd(seed + 2, B, H * G, d, dtype=dtype)
    rec = torch.zeros(B, H, cap // 16, ops.kv4_record_bytes(d), dtype=torch.uint8, device="cuda")
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    bound = bound or max(lens)
    resa.kv4_quantize(dev(k, dtype), dev(v, dtype), bound, rec, H * G, lens=lt)
    clean = rec.cpu().numpy()
    if stale:
        # scales of NaN and codes of ones in every slot past a row's end
        kb, kn, vb, vn, mb = ops._places(d)
        for b, n in enumerate(lens):
            rec[b, :, (n + 15) // 16:] = 0xFF
            for t in range(n, (n + 15) // 16 * 16):
                at = torch.from_numpy(np.concatenate([mb[t % 16] + i for i in range(8)])).cuda()
                rec[b, :, t // 16, at] = 0xFF
                for by, nb in ((kb, kn), (vb, vn)):
                    at = torch.from_numpy(by[t % 16]).cuda()
                    m = torch.from_numpy((15 << (4 * nb[t % 16])).astype(np.uint8)).cuda()
                    for x in (0, 1):
                        w = torch.from_numpy(nb[t % 16] == x).cuda()
                        rec[b, :, t // 16, at[w]] |= m[w]
    qt = dev(q, dtype)
    out = torch.full_like(qt, 7.0)
    lse = torch.full((B, H * G), 7.0, device="cuda")
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, qt), bound)
    scale = 1.0 / math.sqrt(d)
    args = (qt, None, None, rec, None, bound, scale, out, ws)
    resa.decode_dense_kv4(*args, lse=lse, lens=lt)
    assert resa.workspace_status(ws) == resa.RESA_OK
    check(resa, q, clean, lens, None, out.double().cpu().numpy(), lse.double().cpu().numpy(), scale,
          dtype, d, H)
    again = torch.empty_like(out)
    resa.decode_dense_kv4(qt, None, None, rec, None, bound, scale, again, ws, lens=lt)
    assert torch.equal(again, out)                     # no order of arrival shows
    if len(set(lens)) == 1 and bound == lens[0]:
        # without lengths (another cut of the work): the same bounds
        resa.decode_dense_kv4(qt, None, None, rec, None, bound, scale, again, ws, lse=lse)
        check(resa, q, clean, lens, None, again.double().cpu().numpy(), lse.double().cpu().numpy(),
              scale, dtype, d, H)
    return args, out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_below_the_fp32_range_weigh_nothing(resa, dtype):
    # tokens 0 .. 31 (one warp's pair of blocks): logits of -1e39 by a scale of
    # 1000, which q makes up for elsewhere; the others' keys leave channel 0 out
    B, H, G, d, n, scale = 1, 2, 4, 128, 64, 1000.0
    k, v = rnd(1, B, H, n, d, dtype=dtype), rnd(2, B, H, n, d, dtype=dtype)
    q = ops.bf16_round(rnd(3, B, H * G, d) / np.float32(1000 * math.sqrt(d)))
    k[:, :, :, :64], q[:, :, :64] = 0.0, 0.0
    k[:, :, :32, 0], q[:, :, 0] = ops.bf16_round(np.float32(-1e18)), ops.bf16_round(np.float32(1e18))
    rec = torch.zeros(B, H, n // 16, ops.kv4_record_bytes(d), dtype=torch.uint8, device="cuda")
    resa.kv4_quantize(dev(k, dtype), dev(v, dtype), n, rec, H * G)
    qt = dev(q, dtype)
    out, lse = torch.empty_like(qt), torch.empty(B, H * G, device="cuda")
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, qt), n)
    resa.decode_dense_kv4(qt, None, None, rec, None, n, scale, out, ws, lse=lse)
    assert resa.workspace_status(ws) == resa.RESA_OK
    q[:, :, 0] = 0.0
    check(resa, q, rec.cpu().numpy()[:, :, 2:], [32], None, out.double().cpu().numpy(),
          lse.double().cpu().numpy(), scale, dtype, d, H)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 8])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 129, 1000])
def test_dense_decode(resa, dtype, d, G, n):
    run_dense(resa, 2, 2, G, d, dtype, [n, n], (n + 15) // 16 * 16 + 32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,bound", [([1, 700, 33, 16, 2049], None), ([5, 4, 3], 4096),
                                        ([4000] + [1] * 40, None), ([1] * 70, None)])
def test_dense_decode_ragged(resa, dtype, lens, bound):
    run_dense(resa, len(lens), 2, 5, 64, dtype, lens, 4096, bound=bound)


def test_one_head_long_row(resa):
    """One (row, head) split over as many CTAs as a launch may use."""
    run_dense(resa, 1, 1, 4, 128, "bf16", [20011], 20480)


def test_one_long_row_among_short_ones(resa):
    """Nearly every CTA works on one (row, head): more than 64 parts to merge."""
    run_dense(resa, 9, 1, 2, 128, "bf16", [30000] + [3] * 8, 30000)


def test_length_out_of_range_is_clamped_and_flagged(resa):
    k, v = kv_inputs(2, 2, 1, 64, 64, "bf16")
    rec = torch.zeros(2, 1, 4, ops.kv4_record_bytes(64), dtype=torch.uint8, device="cuda")
    resa.kv4_quantize(dev(k, "bf16"), dev(v, "bf16"), 64, rec, 2)
    q = dev(rnd(4, 2, 2, 64), "bf16")
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, q), 64)
    outs = []
    for lens in ([0, 99], [1, 64]):
        out = torch.empty_like(q)
        resa.decode_dense_kv4(q, None, None, rec, None, 64, 0.125, out, ws,
                              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        outs.append(out)
        want = resa.RESA_ERR_BAD_INDEX if lens[0] == 0 else resa.RESA_OK
        assert resa.workspace_status(ws) == want
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_sel", [(1, 1), (300, 5), (2051, 40), (5000, 313)])
def test_attend_blocks(resa, dtype, n, n_sel):
    """Lists in any order; an id out of range is skipped and reported."""
    B, H, G, d, cap = 2, 2, 4, 128, 5008
    k, v = kv_inputs(21, B, H, cap, d, dtype, special=False)
    rec = torch.zeros(B, H, cap // 16, ops.kv4_record_bytes(d), dtype=torch.uint8, device="cuda")
    resa.kv4_quantize(dev(k, dtype), dev(v, dtype), n, rec, H * G)
    q = rnd(9, B, H * G, d, dtype=dtype)
    qt = dev(q, dtype)
    g = np.random.default_rng(3)
    sel = np.stack([np.stack([g.permutation((n + 15) // 16)[:n_sel] for _ in range(H)]) for _ in range(B)])
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, qt), n)
    out, lse = torch.empty_like(qt), torch.empty(B, H * G, device="cuda")
    st = torch.from_numpy(sel.astype(np.int32)).cuda()
    resa.attend_blocks_kv4(qt, rec, n, st, 0.09, out, ws, lse=lse)
    assert resa.workspace_status(ws) == resa.RESA_OK
    check(resa, q, rec.cpu().numpy(), [n] * B, sel, out.double().cpu().numpy(),
          lse.double().cpu().numpy(), 0.09, dtype, d, H)
    if n_sel > 1:
        bad = sel.copy()
        bad[0, 0, 0], bad[1, 1, -1] = -1, (n + 15) // 16
        resa.attend_blocks_kv4(qt, rec, n, torch.from_numpy(bad.astype(np.int32)).cuda(), 0.09, out, ws,
                               lse=lse)
        assert resa.workspace_status(ws) == resa.RESA_ERR_BAD_INDEX
        left = [[sel[0, 0, 1:], sel[0, 1]], [sel[1, 0], sel[1, 1, :-1]]]
        for b in range(B):
            for h in range(H):
                check(resa, q[b:b + 1, h * G:(h + 1) * G], rec[b:b + 1, h:h + 1].cpu().numpy(), [n],
                      np.array([[left[b][h]]]),
                      out[b:b + 1, h * G:(h + 1) * G].double().cpu().numpy(),
                      lse[b:b + 1, h * G:(h + 1) * G].double().cpu().numpy(), 0.09, dtype, d, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[777, 777], [1600, 33, 1]])
def test_sparse_step_is_append_select_attend(resa, dtype, lens):
    """The sparse step selects what select_blocks selects on the exact cache
    (same descriptors) and then attends to those records."""
    B, H, G, d, cap, r, n_min = len(lens), 2, 4, 64, 1600, 0.2, 3
    k, v = kv_inputs(31, B, H, cap, d, dtype, special=False)
    kt, vt = dev(k, dtype), dev(v, dtype)
    ragged = len(set(lens)) > 1
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    prev = torch.clamp(lt - 1, min=1)
    n = max(lens)
    desc = torch.zeros(B, H, cap // 16, 2, d, dtype=DT[dtype], device="cuda")
    resa.build_desc_varlen(kt, prev, n, desc, H * G)
    rec = torch.zeros(B, H, cap // 16, ops.kv4_record_bytes(d), dtype=torch.uint8, device="cuda")
    resa.kv4_quantize(kt, vt, n, rec, H * G, lens=prev)
    q, kn, vn = (dev(rnd(40 + i, B, x, d, dtype=dtype), dtype) for i, x in enumerate((H * G, H, H)))
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, q), n)
    cap_n = resa.num_selected(n, r, n_min)
    sel = torch.full((B, H, cap_n), -9, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B, H * G, device="cuda")
    d2, k2, v2 = desc.clone(), kt.clone(), vt.clone()
    resa.decode_sparse_kv4(q, kn, vn, rec, desc, n, r, n_min, 0.125, out, ws, lse=lse, sel=sel,
                           lens=lt if ragged else None)
    assert resa.workspace_status(ws) == resa.RESA_OK
    ws2 = resa.alloc_workspace(resa.dims_for(k2, H * G), n)
    o2, sel2 = torch.empty_like(q), torch.full_like(sel, -9)
    if ragged:
        resa.decode_sparse_varlen(q, kn, vn, k2, v2, d2, lt, n, r, n_min, 0.125, o2, ws2, sel=sel2)
    else:
        resa.decode_sparse(q, kn, vn, k2, v2, d2, n, r, n_min, 0.125, o2, ws2, sel=sel2)
    assert torch.equal(sel, sel2) and torch.equal(desc, d2)
    rec_np, got, gl = rec.cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    qn, s = q.float().cpu().numpy(), sel.cpu().numpy()
    for b, x in enumerate(lens):
        for h in range(H):
            ids = s[b, h][s[b, h] >= 0]
            check(resa, qn[b:b + 1, h * G:(h + 1) * G], rec_np[b:b + 1, h:h + 1], [x], np.array([[ids]]),
                  got[b:b + 1, h * G:(h + 1) * G], gl[b:b + 1, h * G:(h + 1) * G], 0.125, dtype, d, 1)


def test_graph_replay_other_stream_and_repeatability(resa):
    """A captured call replayed on new queries and lengths, and the same call
    on a side stream, give bit for bit what eager calls give."""
    B, H, G, d, cap = 3, 2, 4, 128, 2048
    args, first = run_dense(resa, B, H, G, d, "bf16", [2048, 2048, 2048], cap)
    q, _, _, rec, _, n, scale, out, ws = args
    lens = torch.tensor([2048, 9, 500], dtype=torch.int32, device="cuda")
    resa.decode_dense_kv4(q, None, None, rec, None, n, scale, out, ws, lens=lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        resa.decode_dense_kv4(q, None, None, rec, None, n, scale, out, ws, lens=lens)
    q.copy_(dev(rnd(77, B, H * G, d), "bf16"))
    lens.copy_(torch.tensor([17, 2048, 1], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    eager = torch.empty_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws2 = resa.alloc_kv4_workspace(resa.dims_kv4(rec, q), n)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        resa.decode_dense_kv4(q, None, None, rec, None, n, scale, eager, ws2, lens=lens)
    side.synchronize()
    assert torch.equal(replayed, eager)
    assert resa.workspace_status(ws) == resa.RESA_OK and resa.workspace_status(ws2) == resa.RESA_OK


@pytest.mark.slow
def test_offsets_past_32_bits(resa):
    """The last rows of a 4.8 GB cache (byte offsets past 2^32)."""
    B, H, G, d, cap, n = 2, 16, 2, 128, 1 << 20, 257
    q = rnd(1, B, H * G, d)
    qt = dev(q, "bf16")
    rec = torch.zeros(B, H, cap // 16, ops.kv4_record_bytes(d), dtype=torch.uint8, device="cuda")
    k, v = kv_inputs(8, 1, 1, 272, d, "bf16", special=False)
    small = torch.zeros(1, 1, 17, ops.kv4_record_bytes(d), dtype=torch.uint8, device="cuda")
    resa.kv4_quantize(dev(k, "bf16"), dev(v, "bf16"), n, small, 2)
    rec[:, :, :17] = small
    out, lse = torch.empty_like(qt), torch.empty(B, H * G, device="cuda")
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, qt), n)
    resa.decode_dense_kv4(qt, None, None, rec, None, n, 0.09, out, ws, lse=lse)
    assert resa.workspace_status(ws) == resa.RESA_OK
    check(resa, q, np.broadcast_to(small.cpu().numpy(), (B, H, 17, small.shape[-1])), [n] * B, None,
          out.double().cpu().numpy(), lse.double().cpu().numpy(), 0.09, "bf16", d, H)


def test_strided_tensors_are_refused(resa):
    rec = torch.zeros(1, 2, 4, ops.kv4_record_bytes(64), dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")[:, :, :64]
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, q), 64)
    with pytest.raises(ValueError):
        resa.decode_dense_kv4(q, None, None, rec, None, 10, 1.0, torch.zeros_like(q), ws)
    k = torch.zeros(1, 2, 64, 128, dtype=torch.bfloat16, device="cuda")[:, :, :, ::2]
    with pytest.raises(ValueError):
        resa.kv4_quantize(k, k, 64, rec, 4)


def test_two_calls_at_once(resa):
    """Two streams, a workspace each: the results of one call after the other."""
    args, out = run_dense(resa, 2, 2, 4, 128, "bf16", [3000, 3000], 3008, stale=False)
    q, _, _, rec, _, n, scale, _, _ = args
    dims = resa.dims_kv4(rec, q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(out) for _ in streams]
    spaces = [resa.alloc_kv4_workspace(dims, n) for _ in streams]
    lens = torch.tensor([3000, 3000], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        for st, o, ws in zip(streams, outs, spaces):
            with torch.cuda.stream(st):
                resa.decode_dense_kv4(q, None, None, rec, None, n, scale, o, ws, lens=lens)
    torch.cuda.synchronize()
    for o, ws in zip(outs, spaces):
        assert torch.equal(o, out) and resa.workspace_status(ws) == resa.RESA_OK


def test_a_model_step_from_packed_prompts_to_a_4_bit_cache(resa):
    """As used together: packed prompts fill the caches and descriptors, the
    caches become 4-bit records, sparse steps append to them."""
    B, H, G, d, cap, lens = 3, 2, 4, 128, 512, [300, 17, 451]
    st = [0, 300, 317, 768]
    T = st[-1]
    q, k, v = (rnd(60 + i, T, x, d) for i, x in enumerate((H * G, H, H)))
    kc = torch.zeros(B, H, cap, d, dtype=torch.bfloat16, device="cuda")
    vc, desc = torch.zeros_like(kc), torch.zeros(B, H, cap // 16, 2, d, dtype=torch.bfloat16, device="cuda")
    qt = dev(q, "bf16")
    out = torch.zeros_like(qt)
    ws = resa.alloc_workspace(resa.dims_for(kc, H * G), cap)
    scale = 1.0 / math.sqrt(d)
    resa.prefill_packed(qt, dev(k, "bf16"), dev(v, "bf16"), torch.tensor(st, dtype=torch.int32, device="cuda"),
                        451, kc, vc, desc, scale, out, ws)
    rec = resa.alloc_kv4(B, H, cap, d)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    resa.kv4_quantize(kc, vc, 451, rec, H * G, lens=lt)
    dq = torch.zeros(B, H * G, d, dtype=torch.bfloat16, device="cuda")
    ws4 = resa.alloc_kv4_workspace(resa.dims_kv4(rec, dq), cap)
    o, lse = torch.zeros_like(dq), torch.zeros(B, H * G, device="cuda")
    for s in range(20):
        qs, kn, vn = (rnd(100 + 3 * s + i, B, x, d) for i, x in enumerate((H * G, H, H)))
        lt += 1
        n = 451 + s + 1
        sel = torch.full((B, H, resa.num_selected(n, 0.3, 4)), -5, dtype=torch.int32, device="cuda")
        resa.decode_sparse_kv4(dev(qs, "bf16"), dev(kn, "bf16"), dev(vn, "bf16"), rec, desc, n, 0.3, 4, scale, o,
                               ws4, lse=lse, sel=sel, lens=lt)
    assert resa.workspace_status(ws4) == resa.RESA_OK and resa.workspace_status(ws) == resa.RESA_OK
    recs, got, gl, ids = rec.cpu().numpy(), o.double().cpu().numpy(), lse.double().cpu().numpy(), sel.cpu().numpy()
    for b in range(B):
        for h in range(H):
            mine = ids[b, h][ids[b, h] >= 0]
            assert len(mine) == resa.num_selected(int(lt[b]), 0.3, 4) and mine[-1] == (int(lt[b]) - 1) // 16
            check(resa, qs[b:b + 1, h * G:(h + 1) * G], recs[b:b + 1, h:h + 1], [int(lt[b])], np.array([[mine]]),
                  got[b:b + 1, h * G:(h + 1) * G], gl[b:b + 1, h * G:(h + 1) * G], scale, "bf16", d, 1)


def dense_both_ways(resa, q, k, v, n, scale, dtype):
    """Outputs and log-sum-exp of a dense step over n quantised tokens, with and
    without row lengths (two cuts of the work), and the records."""
    B, H, cap, d = k.shape
    rec = torch.zeros(B, H, cap // 16, ops.kv4_record_bytes(d), dtype=torch.uint8, device="cuda")
    resa.kv4_quantize(dev(k, dtype), dev(v, dtype), n, rec, q.shape[1])
    qt, res = dev(q, dtype), []
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, qt), n)
    for lens in (None, torch.full((B,), n, dtype=torch.int32, device="cuda")):
        out, lse = torch.empty_like(qt), torch.empty(B, q.shape[1], device="cuda")
        resa.decode_dense_kv4(qt, None, None, rec, None, n, scale, out, ws, lse=lse, lens=lens)
        assert resa.workspace_status(ws) == resa.RESA_OK
        res.append((out.double().cpu().numpy(), lse.double().cpu().numpy()))
    return rec.cpu().numpy(), res


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [32, 8192])
@pytest.mark.parametrize("ramp", [0.0, 5.0, 12.0])
@pytest.mark.parametrize("e", [59, 55, 50, -50])
def test_values_over_their_whole_range(resa, dtype, d, n, ramp, e):
    """Values just below 2^60 (and far below 1): one head's first group constant,
    the others of both signs; equal logits, and logits that grow by `ramp`, so
    that weights pass the running reference by up to 2^8 before it moves."""
    B, H, G = 1, 2, 4
    k = np.zeros((B, H, n, d), np.float32)
    k[..., 0] = ops.bf16_round(np.linspace(0, ramp, n).astype(np.float32))
    v = ops.bf16_round(np.clip(rnd(2, B, H, n, d, dtype=dtype), -1.9, 1.9) * np.float32(2.0 ** e))
    v[:, 0, :, :64] = 2.0 ** e
    q = np.zeros((B, H * G, d), np.float32)
    q[..., 0] = 1.0
    rec, res = dense_both_ways(resa, q, k, v, n, 1.0, dtype)
    for out, lse in res:
        check(resa, q, rec, [n], None, out, lse, 1.0, dtype, d, H)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [3e4, 1e5, 1e6])
def test_large_finite_logits(resa, dtype, size):
    """Queries and keys of 1e4 to 1e6: logits far beyond 2^24, whose rounding is
    wider than any weight's exponent. Where the largest is ahead of the next by
    more than both may be off, the definition gives its value alone."""
    B, H, G, d, n = 2, 2, 4, 128, 300
    scale = 1.0 / math.sqrt(d)
    q = ops.bf16_round(rnd(1, B, H * G, d) * np.float32(size))
    k = ops.bf16_round(rnd(2, B, H, 304, d) * np.float32(size))
    v = rnd(3, B, H, 304, d, dtype=dtype)
    rec, res = dense_both_ways(resa, q, k, v, n, scale, dtype)
    clear = 0
    for b in range(B):
        for g in range(H):
            (kc, ks, kz), (vc, vs, vz) = [tuple(x[:n] for x in y) for y in ops.kv4_unpack(rec[b, g], d)]
            kv, vv = ops.kv4_value(kc, ks, kz), ops.kv4_value(vc, vs, vz)
            for h in range(g * G, g * G + G):
                z = kv @ q[b, h].astype(np.float64) * scale
                # (as in `bounds`, and the rounding to log2 units)
                mag = (np.abs(kz) + 15 * ks).max(-1).max()
                e = (2 * d + 16) * 2.0 ** -24 * scale * np.abs(q[b, h]).sum() * mag + 2.0 ** -22 * np.abs(z).max()
                top = np.sort(z)[-2:]
                for out, lse in res:
                    assert np.isfinite(out[b, h]).all() and abs(lse[b, h] - top[1]) <= e + 6.0
                    if top[1] - top[0] > 2 * e + 100:
                        clear += 1
                        want = vv[z.argmax()]
                        # the code part's rounding, about code 8, and the output's
                        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -21
                        part = 8 * np.repeat(vs[z.argmax()], 64)
                        assert (np.abs(out[b, h] - want) <= half * 1.02 * (part + np.abs(want))).all()
    assert clear >= B * H * G


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_logits_of_any_size(resa, dtype):
    """Heads whose logits are all equal, 2^20 to 2^40 in log2 units: the mean."""
    B, H, G, d, n = 1, 4, 8, 64, 48
    k = np.zeros((B, H, n, d), np.float32)
    k[..., :] = 1024.0                                   # (constant groups are exact)
    v = rnd(3, B, H, n, d, dtype=dtype)
    q = np.zeros((B, H * G, d), np.float32)
    q[0, :, 0] = ops.bf16_round((2.0 ** np.linspace(10, 30, H * G)).astype(np.float32))
    rec, res = dense_both_ways(resa, q, k, v, n, 1.0, dtype)
    for out, lse in res:
        for g in range(H):
            _, (vc, vs, vz) = [tuple(x[:n] for x in y) for y in ops.kv4_unpack(rec[0, g], d)]
            vv = ops.kv4_value(vc, vs, vz)
            want = vv.mean(0)
            # weights of exactly 1 each: roundings of p * scale to bf16 (exact:
            # the scale is bf16), of sums (32 additions) and of the output
            half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
            tol = half * np.abs(want) * 1.02 + 64 * 2.0 ** -23 * (np.abs(vz).max() + 15 * vs.max())
            for h in range(g * G, g * G + G):
                z = 1024.0 * float(q[0, h, 0])
                assert (np.abs(out[0, h] - want) <= tol).all()
                assert abs(lse[0, h] - (z + math.log(n))) <= 2.0 ** -22 * z + 2.0 ** -18
