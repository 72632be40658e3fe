"""The plain definitions of the cache operators (oracle/cache_ops.py), on the CPU."""
import numpy as np
import pytest

from oracle import cache_ops as ops


@pytest.mark.parametrize("d", [64, 128])
def test_record_places_are_a_partition(d):
    """Every nibble and scale byte of a record belongs to exactly one value."""
    kb, kn, vb, vn, mb = ops._places(d)
    ng = d // 64
    for by, nb, lo in ((kb, kn, 0), (vb, vn, 512 * ng)):
        at = set(zip(by.ravel().tolist(), nb.ravel().tolist()))
        assert at == {(lo + i, n) for i in range(512 * ng) for n in (0, 1)}
    assert sorted(mb.ravel().tolist()) == list(range(1024 * ng, ops.kv4_record_bytes(d), 8))


@pytest.mark.parametrize("d", [64, 128])
def test_pack_unpack_round_trip_and_step(d):
    g = np.random.default_rng(1)
    k, v = (ops.bf16_round(g.standard_normal((2, 2, 48, d)).astype(np.float32)) for _ in range(2))
    rec = ops.kv4_pack(k, v, [48, 21])
    for (code, s, z), x in zip(ops.kv4_unpack(rec, d), (k, v)):
        c, sc, ze = ops.kv4_encode(x)
        for b, n in ((0, 48), (1, 21)):
            assert np.array_equal(code[b, :, :n], c[b, :, :n])
            assert np.array_equal(s[b, :, :n], sc[b, :, :n]) and np.array_equal(z[b, :, :n], ze[b, :, :n])
            assert not code[b, :, n:].any() and not s[b, :, n:].any()
        # bf16 data: the zero is exact; half a step, and at the top the scale's
        # own rounding of 15 steps (2^-9 each way, plus fp32 roundings)
        err = np.abs(ops.kv4_value(c, sc, ze) - x)
        step = np.repeat(sc, 64, -1)
        assert (err <= step * (0.5 + 15 * 2.0 ** -8)).all()


def test_constant_groups_have_code_zero():
    c, s, z = ops.kv4_encode(np.full((1, 64), -1.25, np.float32))
    assert not c.any() and not s.any() and (z == -1.25).all()


def test_evict_row_keeps_recent_and_heaviest():
    w = np.array([5, 1, 5, 0, np.nan, 7, -0.0, 2, 9, 9], np.float32)
    assert ops.evict_row(w, 10, 4, 2).tolist() == [0, 5, 8, 9]
    assert ops.evict_row(w, 10, 9, 1).tolist() == [0, 1, 2, 3, 5, 6, 7, 8, 9]
    assert ops.evict_row(w, 10, 10, 1).tolist() == list(range(10))
    tie = np.array([0.0, -0.0, 0.0, 1.0, 1.0], np.float32)
    assert ops.evict_row(tie, 5, 3, 1).tolist() == [0, 3, 4]
