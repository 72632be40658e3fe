"""Boundary checks of the cache operators and packed prompts that need no GPU:
sizes, and every refusal the header promises, before anything is launched."""
import ctypes

import pytest
import torch

FAKE = 0x10000000    # aligned, never dereferenced: validation fails first
STEP = 0x10000000    # between the fake buffers: they do not overlap


@pytest.fixture(scope="module")
def resa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_quest_b200 as m
    return m


def dims(resa, **kw):
    d = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, block_size=16, dtype=resa.RESA_BF16,
             max_len=4096)
    d.update(kw)
    return resa.Dims(**d)


def at(i):
    return FAKE + i * STEP


def test_sizes(resa):
    lib = resa._lib
    d = dims(resa)
    assert resa.kv4_record_bytes(128) == 2304 and resa.kv4_record_bytes(64) == 1152
    assert lib.resa_kv4_bytes(ctypes.byref(d)) == 2 * 2 * 256 * 2304
    assert lib.resa_kv4_bytes(ctypes.byref(dims(resa, head_dim=64))) == 2 * 2 * 256 * 1152
    assert lib.resa_kv4_bytes(ctypes.byref(dims(resa, head_dim=96))) == 0
    sizes = [resa.kv4_workspace_bytes(d, n) for n in (1, 16, 17, 1000, 4096, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and all(s % 256 == 0 for s in sizes)
    logits = [resa.weights_workspace_bytes(d, n) - resa.workspace_bytes(d, n) for n in (1, 1000, 4096)]
    assert logits == sorted(logits) and logits[1] >= 2 * 8 * 1000 * 4
    for f in (lib.resa_kv4_workspace_bytes, lib.resa_weights_workspace_bytes):
        assert f(ctypes.byref(d), 0) == 0 and f(ctypes.byref(dims(resa, block_size=32)), 10) == 0
    with pytest.raises(resa.ResaError):
        resa.kv4_workspace_bytes(d, 0)


def test_kv4_rows_refusals(resa):
    lib, E = resa._lib, resa

    def call(f, d=None, k=at(0), v=at(1), kv4=at(2), n=100, lens=None):
        d = ctypes.byref(d or dims(resa))
        if f == "q":
            return lib.resa_kv4_quantize(d, k, v, n, lens, kv4, None)
        return lib.resa_kv4_dequantize(d, kv4, n, lens, k, v, None)
    for f in "qd":
        for bad in (dict(k=None), dict(v=None), dict(kv4=None), dict(k=at(0) + 8), dict(kv4=at(2) + 4),
                    dict(n=0), dict(lens=at(3) + 2), dict(d=dims(resa, dtype=5))):
            assert call(f, **bad) == E.RESA_ERR_INVALID_ARG, bad
        assert call(f, n=4097) == E.RESA_ERR_CAPACITY
        assert call(f, d=dims(resa, head_dim=96)) == E.RESA_ERR_UNSUPPORTED


def kv4_call(resa, f, d=None, **kw):
    a = dict(q=at(0), kn=None, vn=None, kv4=at(1), desc=at(2), n=100, lens=None, r=0.5, n_min=1, scale=1.0,
             out=at(3), lse=None, sel=at(4), n_sel=3, ws=at(5), wsb=1 << 30)
    a.update(kw)
    d = ctypes.byref(d or dims(resa))
    lib = resa._lib
    if f == "dense":
        return lib.resa_decode_dense_kv4(d, a["q"], a["kn"], a["vn"], a["kv4"], a["desc"], a["n"], a["lens"],
                                         a["scale"], a["out"], a["lse"], a["ws"], a["wsb"], None)
    if f == "sparse":
        return lib.resa_decode_sparse_kv4(d, a["q"], a["kn"], a["vn"], a["kv4"], a["desc"], a["n"], a["lens"],
                                          a["r"], a["n_min"], a["scale"], a["out"], a["lse"], a["sel"], a["ws"],
                                          a["wsb"], None)
    return lib.resa_attend_blocks_kv4(d, a["q"], a["kv4"], a["n"], a["sel"], a["n_sel"], a["scale"], a["out"],
                                      a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("f", ["dense", "sparse", "blocks"])
def test_kv4_decode_refusals(resa, f):
    E = resa
    bad = [dict(q=None), dict(kv4=None), dict(out=None), dict(ws=None), dict(q=at(0) + 4), dict(kv4=at(1) + 8),
           dict(out=at(3) + 2), dict(ws=at(5) + 128), dict(n=0), dict(scale=0.0), dict(scale=-1.0),
           dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e18)]
    if f != "blocks":
        bad += [dict(kn=at(6)), dict(vn=at(6)), dict(kn=at(6) + 4, vn=at(7)), dict(desc=at(2) + 4),
                dict(lens=at(8) + 1)]
    if f == "sparse":
        bad += [dict(desc=None), dict(r=0.0), dict(r=1.5), dict(n_min=0)]
    if f == "blocks":
        bad += [dict(sel=None), dict(n_sel=0), dict(n_sel=8)]
    for b in bad:
        assert kv4_call(resa, f, **b) == E.RESA_ERR_INVALID_ARG, b
    assert kv4_call(resa, f, n=4097) == E.RESA_ERR_CAPACITY
    assert kv4_call(resa, f, wsb=1024) == E.RESA_ERR_WORKSPACE
    need = resa.kv4_workspace_bytes(dims(resa), 100)
    assert kv4_call(resa, f, wsb=need - 1) == E.RESA_ERR_WORKSPACE
    assert kv4_call(resa, f, d=dims(resa, n_q_heads=18)) == E.RESA_ERR_UNSUPPORTED
    assert kv4_call(resa, f, d=dims(resa, n_q_heads=7)) == E.RESA_ERR_INVALID_ARG


def test_sparse_kv4_refuses_more_blocks_than_a_selection_takes(resa):
    d = dims(resa, batch=1, n_q_heads=1, n_kv_heads=1, max_len=16 * 262145)
    assert kv4_call(resa, "sparse", d=d, n=16 * 262144 + 1) == resa.RESA_ERR_UNSUPPORTED


@pytest.mark.parametrize("f", ["dense", "sparse", "blocks"])
def test_kv4_refuses_more_heads_than_its_work_split_can_number(resa, f):
    # 65535 x 1024 heads of one block: 65 positions each, more than 2^32 in all
    d = dims(resa, batch=65535, n_q_heads=1024, n_kv_heads=1024, max_len=16)
    assert kv4_call(resa, f, d=d, n=16, n_sel=1, wsb=1 << 60) == resa.RESA_ERR_UNSUPPORTED


def test_weights_refusals(resa):
    lib, E = resa._lib, resa

    def call(d=None, **kw):
        a = dict(q=at(0), kn=None, vn=None, k=at(1), v=at(2), desc=at(3), w=at(4), n=100, lens=None, scale=1.0,
                 out=at(5), lse=None, ws=at(6), wsb=1 << 30)
        a.update(kw)
        return lib.resa_decode_dense_weights(ctypes.byref(d or dims(resa)), a["q"], a["kn"], a["vn"], a["k"],
                                             a["v"], a["desc"], a["w"], a["n"], a["lens"], a["scale"], a["out"],
                                             a["lse"], a["ws"], a["wsb"], None)
    for b in (dict(q=None), dict(k=None), dict(v=None), dict(w=None), dict(w=at(4) + 4), dict(out=None),
              dict(ws=None), dict(ws=at(6) + 64), dict(kn=at(7)), dict(desc=at(3) + 8), dict(lens=at(8) + 3),
              dict(n=0), dict(scale=0.0), dict(scale=float("nan"))):
        assert call(**b) == E.RESA_ERR_INVALID_ARG, b
    assert call(n=4097) == E.RESA_ERR_CAPACITY
    # a workspace for the plain step does not hold the logits
    assert call(wsb=resa.workspace_bytes(dims(resa), 100)) == E.RESA_ERR_WORKSPACE
    assert call(d=dims(resa, head_dim=32)) == E.RESA_ERR_UNSUPPORTED


def test_evict_refusals(resa):
    lib, E = resa._lib, resa

    def call(d=None, **kw):
        a = dict(k=at(0), v=at(1), w=at(2), n=1000, lens=None, budget=100, recent=10, lo=112, ko=at(3), vo=at(4),
                 do=at(5), wo=at(6), kept=at(7), ws=at(8), wsb=1 << 30)
        a.update(kw)
        return lib.resa_evict(ctypes.byref(d or dims(resa)), a["k"], a["v"], a["w"], a["n"], a["lens"], a["budget"],
                              a["recent"], a["lo"], a["ko"], a["vo"], a["do"], a["wo"], a["kept"], a["ws"],
                              a["wsb"], None)
    for b in (dict(k=None), dict(v=None), dict(w=None), dict(ko=None), dict(vo=None), dict(kept=None),
              dict(ws=None), dict(k=at(0) + 4), dict(w=at(2) + 4), dict(vo=at(4) + 4), dict(do=at(5) + 4),
              dict(wo=at(6) + 2), dict(kept=at(7) + 2), dict(lens=at(9) + 2), dict(n=0), dict(budget=0),
              dict(recent=-1), dict(recent=101), dict(lo=100), dict(lo=0),
              # outputs on inputs, or on each other
              dict(ko=at(0)), dict(vo=at(0) + 4096), dict(wo=at(2) + 16), dict(do=at(1)), dict(kept=at(2)),
              dict(vo=at(3) + 1024), dict(do=at(3)), dict(kept=at(6))):
        assert call(**b) == E.RESA_ERR_INVALID_ARG, b
    assert call(n=4097) == E.RESA_ERR_CAPACITY
    assert call(budget=113) == E.RESA_ERR_CAPACITY
    assert call(wsb=64) == E.RESA_ERR_WORKSPACE
    assert call(d=dims(resa, head_dim=96)) == E.RESA_ERR_UNSUPPORTED


def test_packed_refusals(resa):
    lib, E = resa._lib, resa

    def call(d=None, **kw):
        a = dict(q=at(0), k=at(1), v=at(2), st=at(3), total=500, longest=300, kc=at(4), vc=at(5), desc=at(6),
                 scale=1.0, out=at(7), ws=at(8), wsb=1 << 20)
        a.update(kw)
        return lib.resa_prefill_packed(ctypes.byref(d or dims(resa)), a["q"], a["k"], a["v"], a["st"], a["total"],
                                       a["longest"], a["kc"], a["vc"], a["desc"], a["scale"], a["out"], a["ws"],
                                       a["wsb"], None)
    for b in (dict(q=None), dict(k=None), dict(v=None), dict(st=None), dict(out=None), dict(ws=None),
              dict(kc=None), dict(vc=None), dict(q=at(0) + 8), dict(k=at(1) + 2), dict(out=at(7) + 4),
              dict(kc=at(4) + 8), dict(desc=at(6) + 2), dict(st=at(3) + 1), dict(ws=at(8) + 16), dict(total=0),
              dict(longest=0), dict(scale=0.0), dict(scale=float("inf")), dict(out=at(0)), dict(out=at(1) + 1024),
              dict(kc=at(1)), dict(vc=at(2) + 512), dict(desc=at(0)), dict(vc=at(4) + 4096), dict(desc=at(5))):
        assert call(**b) == E.RESA_ERR_INVALID_ARG, b
    assert call(longest=4097) == E.RESA_ERR_CAPACITY
    assert call(wsb=128) == E.RESA_ERR_WORKSPACE
    assert call(d=dims(resa, dtype=resa.RESA_F32)) == E.RESA_ERR_UNSUPPORTED
    assert call(d=dims(resa, head_dim=256)) == E.RESA_ERR_UNSUPPORTED
    assert call(total=2**31) == E.RESA_ERR_UNSUPPORTED


def test_binding_refuses_what_the_library_cannot_see(resa):
    """Wrong shapes, types and devices (here: the CPU) are refused in Python."""
    q = torch.zeros(1, 4, 64)
    kv4 = torch.zeros(1, 2, 3, 1152, dtype=torch.uint8)
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError):
        resa.dims_kv4(kv4, torch.zeros(1, 4, 128))
    with pytest.raises(ValueError):
        resa.dims_kv4(kv4.view(torch.int8), q)
    for out, lse, kn in ((torch.zeros(1, 4, 32), None, None), (q, torch.zeros(3), None),
                         (q, None, torch.zeros(1, 4, 64)), (q.bfloat16(), None, None)):
        with pytest.raises(ValueError):
            resa.decode_dense_kv4(q, kn, kn, kv4, None, 10, 1.0, out, ws, lse=lse)
    k = torch.zeros(1, 2, 48, 64)
    with pytest.raises(ValueError):
        resa.kv4_quantize(k, k, 10, kv4[:, :, :2], 4)
    with pytest.raises(ValueError):
        resa.decode_dense_weights(q, None, None, k, k, None, torch.zeros(1, 2, 47), 10, 1.0, q, None, ws)
    with pytest.raises(ValueError):
        resa.evict(k, k, torch.zeros(1, 2, 48), 10, 5, 1, torch.zeros(1, 2, 16, 32), k, None, None,
                   torch.zeros(1, 2, 5, dtype=torch.int32), 4, ws)


def test_tensors_of_the_cpu_are_refused(resa):
    """No address of host memory reaches a kernel, whether all tensors of a call
    or some of them lie there."""
    def z(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype)

    q, k, ws = z(1, 4, 64), z(1, 2, 48, 64), z(1 << 20, dtype=torch.uint8)
    kv4, lens = z(1, 2, 3, 1152, dtype=torch.uint8), z(1, dtype=torch.int32)
    sel, w = z(1, 2, 2, dtype=torch.int32), z(1, 2, 48)
    calls = [lambda: resa._ptrs(q), lambda: resa._ptrs(None, q, k),
             lambda: resa.kv4_quantize(k, k, 10, kv4, 4),
             lambda: resa.kv4_dequantize(kv4, 10, k, k, 4, lens=lens),
             lambda: resa.decode_dense_kv4(q, None, None, kv4, None, 10, 1.0, z(1, 4, 64), ws),
             lambda: resa.decode_sparse_kv4(q, None, None, kv4, z(1, 2, 3, 2, 64), 48, 0.5, 1, 1.0, z(1, 4, 64), ws),
             lambda: resa.attend_blocks_kv4(q, kv4, 48, sel, 1.0, z(1, 4, 64), ws),
             lambda: resa.decode_dense_weights(q, None, None, k, k, None, w, 10, 1.0, z(1, 4, 64), None, ws),
             lambda: resa.evict(k, k, w, 10, 5, 1, z(1, 2, 16, 64), z(1, 2, 16, 64), None, None,
                                z(1, 2, 5, dtype=torch.int32), 4, ws),
             lambda: resa.prefill_packed(z(9, 4, 64), z(9, 2, 64), z(9, 2, 64), z(2, dtype=torch.int32), 9, k, k, None,
                                         1.0, z(9, 4, 64), ws)]
    for f in calls:
        with pytest.raises(ValueError, match="CUDA device"):
            f()


def test_packed_prompts_without_caches_are_checked_like_others(resa):
    """Caches may be left out (both); what is left is checked all the same."""
    q, k, st = torch.zeros(9, 4, 64), torch.zeros(9, 2, 64), torch.zeros(3, dtype=torch.int32)
    c, desc, ws = torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 1, 2, 64), torch.zeros(1024, dtype=torch.uint8)
    for kw, what in ((dict(), "CUDA"), (dict(ds=None), "CUDA"), (dict(kc=c, vc=c), "CUDA"),
                     (dict(kc=c), "both"), (dict(vc=c), "both"), (dict(ds=desc[:1]), "desc"), (dict(ds=desc[0]), "desc"),
                     (dict(kc=c[:1], vc=c[:1]), "caches"), (dict(kc=c, vc=c.bfloat16()), "dtype"),
                     (dict(st=st[:1]), "starts"), (dict(st=st.long()), "starts"), (dict(k=k[:8]), "total")):
        a = dict(dict(k=k, st=st, kc=None, vc=None, ds=desc), **kw)
        with pytest.raises(ValueError, match=what):
            resa.prefill_packed(q, a["k"], k, a["st"], 9, a["kc"], a["vc"], a["ds"], 1.0, torch.zeros_like(q), ws)


def test_misaligned_results_are_refused(resa):
    """lse and sel are written (sel also read) four bytes at a time. (The
    workspace is too small throughout: no call gets as far as a launch.)"""
    E = resa
    for f in ("dense", "sparse", "blocks"):
        assert kv4_call(resa, f, lse=at(6) + 2, wsb=64) == E.RESA_ERR_INVALID_ARG, f
        assert kv4_call(resa, f, lse=at(6) + 4, wsb=64) == E.RESA_ERR_WORKSPACE, f
    for f in ("sparse", "blocks"):
        assert kv4_call(resa, f, sel=at(4) + 1, wsb=64) == E.RESA_ERR_INVALID_ARG, f
    d, small = ctypes.byref(dims(resa)), resa.workspace_bytes(dims(resa), 100)
    for lse, want in ((at(6) + 2, E.RESA_ERR_INVALID_ARG), (at(6) + 4, E.RESA_ERR_WORKSPACE)):
        rc = resa._lib.resa_decode_dense_weights(d, at(0), None, None, at(1), at(2), None, at(3), 100, None, 1.0, at(4),
                                                 lse, at(5), small, None)
        assert rc == want
