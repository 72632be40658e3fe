"""fp32 calls on the 4-bit cache keep 24 bits of q and of p * scale.

The bounds in test_gpu_kv4.py hold for any order of fp32 sums and are too wide
to tell three bf16 parts from two. Here the inputs leave almost no rounding but
the parts', and the bounds are a few units u = 2^-24. On the CPU, the same
inputs with two parts have to miss them."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_ops as ops

U = 2.0 ** -24


@pytest.fixture(scope="module")
def resa():
    import __graft_entry__
    __graft_entry__.build()
    import block_sparse_attention_quest_b200 as m
    return m


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()


def parts(x, n):
    """Sum of the first n bf16 parts of fp32 x (each the rounding of what is left)."""
    x = np.asarray(x, np.float32)
    got = np.zeros(x.shape, np.float64)
    for _ in range(n):
        p = ops.bf16_round(x)
        got += p
        x = x - p
    return got


# ------------------------------------------------------------------ parts of q
#
# One token: its logit is the log-sum-exp. Keys of 15 (or -15) and 0 in turn, so
# scale 1 and codes 15 and 0; q = x 2^e in every channel, with x = 1 + 2^-9 +
# 2^-17 - 2^-23: parts 1, 2^-9 and 2^-17 - 2^-23, whose loss moves the logit by
# 2^-17 = 128 u of itself. With three parts: in each group of 64 channels, four
# products of first parts truncated at 2 u each at most (the other parts' sums
# are smaller by 2^9), the factors, zero and sum of groups 6 u, the scale, the
# softmax scale (1/128) and log2 units 2 u, back to natural units 2 u, the two
# terms of a logit (7 or 8 of 15 each) of one sign.
Q_BOUND = (8 + 6 + 2 + 2) * U
X = 1 + 2.0 ** -9 + 2.0 ** -17 - 2.0 ** -23


def q_case(d):
    q = np.zeros((1, 16, d), np.float32)
    q[0] = X * 2.0 ** np.linspace(-4, 3, 16).round()[:, None]
    k = np.zeros((1, 2, 16, d), np.float32)
    k[0, 0, :, ::2], k[0, 1, :, 1::2] = 15.0, -15.0
    z = np.einsum("hd,hd->h", q[0].astype(np.float64), k[0, :, 0].astype(np.float64).repeat(8, 0)) / 128
    return q, k, z


@pytest.mark.parametrize("d", [64, 128])
def test_two_parts_of_q_would_be_seen(d):
    q, k, z = q_case(d)
    assert np.array_equal(parts(q, 3), q.astype(np.float64))
    two = np.einsum("hd,hd->h", parts(q, 2)[0], k[0, :, 0].astype(np.float64).repeat(8, 0)) / 128
    assert (np.abs(two - z) > 4 * Q_BOUND * np.abs(z)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("blocks", [False, True])
def test_parts_of_q(resa, d, blocks):
    q, k, z = q_case(d)
    _, lse = attend(resa, q, k, np.zeros_like(k), 1, 1.0 / 128, blocks)
    assert (np.abs(lse[0] - z) <= Q_BOUND * np.abs(z)).all(), np.abs(lse[0] / z - 1).max() / U


# ------------------------------------------------------- parts of p * scale
#
# One block: token 0 with logit 0 and value 0, fifteen with logit -15 q_0 and
# values 7 and -8 in turn (scale 1, zero -8: zero + 8 scale is 0 and p * scale
# is p). The output is 15 p {7, -8} / (1 + 15 p). Parts of p lost are lost from
# the numerator alone. With three: two of the three products that add up to a
# block truncated at 2 u, 1 u for the running sum, 5 u for the sum of weights (two
# additions and three shuffles of a lane's), 1 u for its reciprocal, 1 u for the
# product with it; p's own error (exp2 2^-22, its argument 4 u of at most 1)
# enters divided by 1 + 15 p > 8.
P_BOUND = (4 + 1 + 5 + 1 + 1 + 2) * U


def p_case(d):
    H, G = 8, 8
    q = np.zeros((1, H * G, d), np.float32)
    q[0, :, 0] = np.linspace(0.004, 0.046, H * G).astype(np.float32)
    k, v = np.zeros((1, H, 16, d), np.float32), np.zeros((1, H, 16, d), np.float32)
    k[:, :, 1:, 0] = -15.0
    v[:, :, 1:, ::2], v[:, :, 1:, 1::2] = 7.0, -8.0
    p = np.exp(-15.0 * q[0, :, 0].astype(np.float64))
    sign = np.where(np.arange(d) % 2 == 0, 7.0, -8.0)
    return q, k, v, p, sign


def test_two_parts_of_p_would_be_seen():
    _, _, _, p, sign = p_case(128)
    p = p.astype(np.float32)
    assert np.abs(parts(p, 3) / p - 1).max() <= U
    lost = np.abs(parts(p, 2) / p - 1)                 # of the output, relatively
    assert (lost > P_BOUND).mean() > 0.5 and lost.max() > 4 * P_BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("blocks", [False, True])
def test_parts_of_p(resa, d, blocks):
    q, k, v, p, sign = p_case(d)
    out, lse = attend(resa, q, k, v, 16, 1.0, blocks)
    want = (15 * p / (1 + 15 * p))[:, None] * sign
    assert (np.abs(out[0] - want) <= P_BOUND * np.abs(want)).all(), np.abs(out[0] / want - 1).max() / U


def attend(resa, q, k, v, n, scale, blocks):
    B, H, cap, d = k.shape
    rec = resa.alloc_kv4(B, H, cap, d)
    resa.kv4_quantize(dev(k), dev(v), n, rec, q.shape[1])
    qt = dev(q)
    out, lse = torch.empty_like(qt), torch.empty(B, q.shape[1], device="cuda")
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, qt), n)
    if blocks:
        sel = torch.arange((n + 15) // 16, dtype=torch.int32, device="cuda").expand(B, H, -1).contiguous()
        resa.attend_blocks_kv4(qt, rec, n, sel, scale, out, ws, lse=lse)
    else:
        resa.decode_dense_kv4(qt, None, None, rec, None, n, scale, out, ws, lse=lse)
    assert resa.workspace_status(ws) == resa.RESA_OK
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


# ----------------------------------------------------------------- long sums
#
# Keys and values with a common part per channel, over which truncated sums
# drift. The reference is 64-bit attention over the same records; the measure
# the same in plain 32-bit torch operations, which adds the same terms: their
# worst outputs over a hundred heads of one distribution are of one size, and
# the kernel may be at most four times as far off (sums that truncated instead
# of rounding, or products of codes about 0, were ten times as far).

@pytest.mark.gpu
@pytest.mark.parametrize("n,blocks", [(1000, False), (32001, False), (32001, True)])
def test_long_sums_are_as_exact_as_plain_fp32(resa, n, blocks):
    B, H, G, d = 4, 16, 4, 128                         # (two CTAs per head: long sums per warp)
    cap, scale = (n + 15) // 16 * 16, 1.0 / math.sqrt(128)
    g = torch.Generator(device="cuda").manual_seed(5)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    k, v, q = randn(B, H, cap, d), randn(B, H, cap, d), randn(B, H * G, d)
    k += 0.5 * randn(1, H, 1, d)
    v += 1.5
    rec = resa.alloc_kv4(B, H, cap, d)
    resa.kv4_quantize(k, v, n, rec, H * G)
    out, lse = torch.empty_like(q), torch.empty(B, H * G, device="cuda")
    ws = resa.alloc_kv4_workspace(resa.dims_kv4(rec, q), n)
    if blocks:
        sel = torch.arange(cap // 16, dtype=torch.int32, device="cuda").expand(B, H, -1).contiguous()
        resa.attend_blocks_kv4(q, rec, n, sel, scale, out, ws, lse=lse)
    else:
        resa.decode_dense_kv4(q, None, None, rec, None, n, scale, out, ws, lse=lse)
    assert resa.workspace_status(ws) == resa.RESA_OK
    assert not torch.backends.cuda.matmul.allow_tf32
    far = {"out": [0.0, 0.0], "lse": [0.0, 0.0]}
    for b in range(B):
        for h in range(0, H, 2):
            (kc, ks, kz), (vc, vs, vz) = [tuple(x[:n] for x in y) for y in ops.kv4_unpack(rec[b, h].cpu().numpy(), d)]
            kk, vv = (torch.from_numpy(ops.kv4_value(*x)).cuda() for x in ((kc, ks, kz), (vc, vs, vz)))
            qq = q[b, h * G:(h + 1) * G]
            z = qq.double() @ kk.t() * scale
            e = torch.logsumexp(z, -1)
            ref = torch.exp(z - e.unsqueeze(-1)) @ vv
            z32 = qq @ kk.float().t() * scale
            top = z32.amax(-1, keepdim=True)
            p32 = torch.exp(z32 - top)
            l32 = p32.sum(-1, keepdim=True)
            plain, e32 = (p32 / l32) @ vv.float(), (top + torch.log(l32))[:, 0]
            for name, got, base, want in (("out", out[b, h * G:(h + 1) * G], plain, ref),
                                          ("lse", lse[b, h * G:(h + 1) * G], e32, e)):
                far[name][0] = max(far[name][0], float((got.double() - want).abs().max()))
                far[name][1] = max(far[name][1], float((base.double() - want).abs().max()))
    print(n, blocks, far)
    for name, (got, plain) in far.items():
        assert got <= 4 * plain, (name, far)
