"""Plain CPU definitions of the cache operators beside the block-sparse decode:
the 4-bit cache, attention weights and eviction, packed prompts.

TEST INFRASTRUCTURE, as resa_oracle.py: NumPy, written from the definitions in
include/resa.h, sharing no code with the CUDA library. Arithmetic is float64
except where a definition fixes fp32 (which code, scale and zero a value gets).
"""
from __future__ import annotations

import numpy as np

BLOCK = 16
GROUP = 64


def bf16_round(x: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest, ties to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


# ------------------------------------------------------------- the 4-bit cache

def kv4_encode(x: np.ndarray):
    """x [..., d] fp32 -> codes [..., d] uint8, scale and zero [..., d / 64] fp32."""
    y = np.asarray(x, np.float32)
    y = y.reshape(*y.shape[:-1], -1, GROUP)
    lo, hi = y.min(-1), y.max(-1)
    scale = bf16_round((hi - lo) * np.float32(1.0 / 15.0))
    zero = bf16_round(lo)
    safe = np.where(scale > 0, scale, np.float32(1.0))[..., None]
    q = np.rint((y - zero[..., None]) / safe)
    code = np.where(scale[..., None] > 0, np.clip(q, 0, 15), 0)
    return code.astype(np.uint8).reshape(x.shape), scale, zero


def kv4_value(code, scale, zero) -> np.ndarray:
    """zero + scale * code in float64."""
    c = code.reshape(*code.shape[:-1], -1, GROUP).astype(np.float64)
    v = zero[..., None].astype(np.float64) + scale[..., None].astype(np.float64) * c
    return v.reshape(code.shape)


def kv4_record_bytes(d: int) -> int:
    return BLOCK * (d + 8 * (d // GROUP))


def _places(d: int):
    """Byte of a record and nibble of it for every (token, channel) of keys and
    of values, and the byte of every (token, group)'s scales."""
    ng = d // GROUP
    kb, vb = np.zeros((BLOCK, d), int), np.zeros((BLOCK, d), int)
    kn, vn = np.zeros((BLOCK, d), int), np.zeros((BLOCK, d), int)
    mb = np.zeros((BLOCK, ng), int)
    for t in range(BLOCK):
        for ch in range(d):
            g, x = divmod(ch, GROUP)
            # key: token 8h + r, channel 16c + 8j + i: nibble i of word [g][r][c][2h + j]
            h, r = divmod(t, 8)
            c, rest = divmod(x, 16)
            j, i = divmod(rest, 8)
            word = ((g * 8 + r) * 4 + c) * 4 + 2 * h + j
            kb[t, ch], kn[t, ch] = 4 * word + i // 2, i % 2
            # value: token 8h + 2c + o, channel 16m + 8e + r: nibble e + 2h + 4o of [g][r][c][m]
            c, o = divmod(t % 8, 2)
            m, rest = divmod(x, 16)
            e, r = divmod(rest, 8)
            word = ((g * 8 + r) * 4 + c) * 4 + m
            nib = e + 2 * h + 4 * o
            vb[t, ch], vn[t, ch] = 512 * ng + 4 * word + nib // 2, nib % 2
        for g in range(ng):
            mb[t, g] = 1024 * ng + (((t % 8) * 2 + t // 8) * ng + g) * 8
    return kb, kn, vb, vn, mb


def _bf16_bytes(x: np.ndarray) -> np.ndarray:
    u = (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.stack([u & 255, u >> 8], -1).astype(np.uint8)


def kv4_pack(k: np.ndarray, v: np.ndarray, lens) -> np.ndarray:
    """Records [B, H, L/16, bytes] of the first lens[b] tokens of k, v [B, H, L, d];
    bytes of slots past a row's end are zero."""
    B, H, L, d = k.shape
    ng = d // GROUP
    kb, kn, vb, vn, mb = _places(d)
    rec = np.zeros((B, H, L // BLOCK, kv4_record_bytes(d)), np.uint8)
    for b in range(B):
        n = int(lens[b])
        enc = [kv4_encode(x[b, :, :n]) for x in (k, v)]
        for t in range(n):
            j, s = divmod(t, BLOCK)
            for (code, scale, zero), by, nb, off in ((enc[0], kb, kn, 0), (enc[1], vb, vn, 4)):
                for hh in range(H):
                    np.bitwise_or.at(rec[b, hh, j], by[s], code[hh, t] << (4 * nb[s]).astype(np.uint8))
                    for g in range(ng):
                        at = mb[s, g] + off
                        rec[b, hh, j, at:at + 2] = _bf16_bytes(scale[hh, t, g])
                        rec[b, hh, j, at + 2:at + 4] = _bf16_bytes(zero[hh, t, g])
    return rec


def kv4_unpack(rec: np.ndarray, d: int):
    """Codes, scales and zeros of keys, then of values: each [..., L, d] or [..., L, d/64]."""
    ng = d // GROUP
    kb, kn, vb, vn, mb = _places(d)
    lead = rec.shape[:-2]
    out = []
    for by, nb, off in ((kb, kn, 0), (vb, vn, 4)):
        code = (rec[..., by] >> (4 * nb).astype(np.uint8)) & 15
        sc = []
        for o in (0, 2):
            lo, hi = rec[..., mb + off + o].astype(np.uint32), rec[..., mb + off + o + 1].astype(np.uint32)
            sc.append(np.ascontiguousarray((lo | hi << 8) << 16).view(np.float32))
        out.append((code.reshape(*lead, -1, d), sc[0].reshape(*lead, -1, ng), sc[1].reshape(*lead, -1, ng)))
    return out


# ------------------------------------------------------------------- attention

def attend_row(q, k, v, scale):
    """Heads q [G, d] over k, v [n, d]: outputs, natural log-sum-exp, weights [G, n]."""
    z = np.asarray(q, np.float64) @ np.asarray(k, np.float64).T * scale
    top = z.max(-1, keepdims=True)
    e = np.exp(z - top)
    tot = e.sum(-1, keepdims=True)
    w = e / tot
    return w @ np.asarray(v, np.float64), (top + np.log(tot))[:, 0], w


# -------------------------------------------------------------------- eviction

def evict_row(w: np.ndarray, n: int, budget: int, recent: int) -> np.ndarray:
    """Kept tokens (ascending) of one KV head: the last `recent` and, of the
    others, the budget - recent of the largest weight (NaN below every number,
    -0 equal to +0, ties to the lower index)."""
    if n <= budget:
        return np.arange(n)
    x = np.asarray(w[:n - recent], np.float64)
    key = np.where(np.isnan(x), -np.inf, x)
    order = np.lexsort((np.arange(n - recent), np.isnan(x), -key))
    return np.concatenate([np.sort(order[:budget - recent]), np.arange(n - recent, n)])


def descriptors(k: np.ndarray, n: int):
    """Per-block per-channel minimum and maximum [ceil(n/16), 2, d] of k [>= n, d]."""
    out = []
    for t in range(0, n, BLOCK):
        blk = k[t:min(n, t + BLOCK)]
        out.append(np.stack([blk.min(0), blk.max(0)]))
    return np.stack(out) if out else np.zeros((0, 2, k.shape[-1]))


# -------------------------------------------------------------- packed prompts

def packed_causal(q, k, v, starts, scale):
    """q [T, Hq, d], k, v [T, H, d]: causal attention inside every sequence
    starts[i] .. starts[i + 1] - 1; NaN rows behind the last one."""
    G = q.shape[1] // k.shape[1]
    out = np.full(q.shape, np.nan)
    for a, e in zip(starts[:-1], starts[1:]):
        n = e - a
        for h in range(q.shape[1]):
            z = q[a:e, h].astype(np.float64) @ k[a:e, h // G].astype(np.float64).T * scale
            z = np.where(np.tril(np.ones((n, n), bool)), z, -np.inf)
            if n:
                z -= z.max(-1, keepdims=True)
                p = np.exp(z)
                out[a:e, h] = (p / p.sum(-1, keepdims=True)) @ v[a:e, h // G].astype(np.float64)
    return out
