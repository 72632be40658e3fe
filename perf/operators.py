"""The smaller-cache and packed-prompt operators of this library, as measured.

Five operators next to the block-sparse decode they serve:

* ``quantize``  a prompt's bf16 or fp32 keys and values written into a 4-bit
                cache, and read back as the values that cache stands for;
* ``kv4``       one decode step's attention over a 4-bit cache, over all of a
                row's tokens or over a list of its 16-token blocks;
* ``weights``   a dense decode step that also adds every key's attention
                weight to a running sum;
* ``evict``     a cache cut to the tokens that gathered the most weight;
* ``packed``    causal attention over packed prompts of different lengths,
                which fills the caches and block descriptors to decode from.

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits; where it is true, with the library's calls. ``exact`` computes the
same outputs in 64 bits from the definitions.
"""
import math

import torch

own = False

BLOCK = 16                 # tokens of a block, and of a record of the 4-bit cache
GROUP = 64                 # channels that share one scale and zero point
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    h = {"hq": 32, "hk": 8, "d": 128, "dtype": "bf16"}
    return [
        # a short prompt's cache moved to 4 bits before its first decode step
        {"name": "quantize_2k", "op": "quantize", "b": 1, "len": 2111, **h},
        # a long document's cache moved to 4 bits
        {"name": "quantize_128k", "op": "quantize", "b": 1, "len": 131072, **h},
        # the first steps of a chat: latency alone counts
        {"name": "kv4_chat_start", "op": "kv4", "b": 1, "len": 33, "ragged": False, "r": 1.0,
         "hq": 8, "hk": 2, "d": 64, "dtype": "f32"},
        # one step over a whole 128K context in 4 bits
        {"name": "kv4_dense_128k", "op": "kv4", "b": 1, "len": 131072, "ragged": False, "r": 1.0, **h},
        # one block-sparse step over a 256K context, a tenth of its blocks
        {"name": "kv4_sparse_256k", "op": "kv4", "b": 1, "len": 262139, "ragged": False, "r": 0.1, **h},
        # a serving batch of conversations of different lengths
        {"name": "kv4_ragged_batch", "op": "kv4", "b": 16, "len": 32768, "ragged": True, "r": 1.0, **h},
        # weight bookkeeping early in a conversation, fp32 cache
        {"name": "weights_1k", "op": "weights", "b": 2, "len": 1000, "ragged": True,
         "hq": 16, "hk": 4, "d": 64, "dtype": "f32"},
        # weight bookkeeping of one step over a 128K context
        {"name": "weights_128k", "op": "weights", "b": 1, "len": 131072, "ragged": False, **h},
        # a small cache cut back to its budget
        {"name": "evict_4k", "op": "evict", "b": 2, "len": 4097, "budget": 1001, "recent": 65,
         "hq": 16, "hk": 4, "d": 64, "dtype": "f32"},
        # a 128K cache cut to an eighth
        {"name": "evict_128k", "op": "evict", "b": 1, "len": 131072, "budget": 16384, "recent": 512, **h},
        # a batch of short requests arriving together
        {"name": "packed_short", "op": "packed", "b": 24, "total": 2500, **h},
        # a few long documents prefilled in one call
        {"name": "packed_32k", "op": "packed", "b": 3, "total": 32768, **h},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "kv4", "weights", "evict", "packed"])
    hk = rng.choice([1, 2, 4, 8])
    g = rng.choice([x for x in ([1, 2, 4, 8] if op == "packed" else [1, 2, 4, 5, 8]) if x * hk <= 40])
    c = {"op": op, "hq": hk * g, "hk": hk, "d": rng.choice([64, 128]),
         "dtype": "bf16" if op == "packed" else rng.choice(["bf16", "bf16", "f32"])}
    b = rng.choice([1, 1, 2, 3, 7])
    if op == "packed":
        c["b"] = rng.choice([1, 2, 5, 16, 33])
        c["total"] = _log(rng, 64, 16000)
        return c
    c["b"] = b
    c["len"] = _log(rng, 17, (131072 if c["dtype"] == "bf16" else 65536) // b)
    if op == "kv4":
        c["ragged"] = rng.random() < 0.5
        c["r"] = 1.0 if c["ragged"] else rng.choice([1.0, 0.3, 0.1])
    if op == "weights":
        c["ragged"] = rng.random() < 0.5
    if op == "evict":
        c["len"] = max(64, c["len"])
        c["budget"] = _log(rng, 33, c["len"])
        c["recent"] = rng.randint(1, c["budget"] // 2)
    return c


def _capacity(n):
    return (n + BLOCK - 1) // BLOCK * BLOCK


def _ragged_lengths(case):
    """Row lengths between an eighth of `len` and `len`, the last one `len`."""
    b, n = case["b"], case["len"]
    if not case.get("ragged"):
        return [n] * b
    return [max(1, n * (2 * i + 1 + (b < 2) * b) // (2 * b) + i % 3) for i in range(b - 1)] + [n]


def _packed_lengths(case):
    """Sequence lengths that sum to `total`: one about half of it, the others
    uneven, an empty one among many."""
    b, total = case["b"], case["total"]
    if b == 1:
        return [total]
    rest = total - total // 2
    w = [(7 * i) % 11 + 1 for i in range(b - 1)]
    if b > 4:
        w[2] = 0
    cut = [rest * x // sum(w) for x in w]
    cut[0] += rest - sum(cut)
    return cut[:1] + [total // 2] + cut[1:]


def _selected(case):
    m = (case["len"] + BLOCK - 1) // BLOCK
    return min(m, max(4, math.ceil(m * case["r"])))


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _cache(g, b, hk, n, d, dtype, cap):
    """Keys and values of n tokens in a cache of `cap`; keys with an offset per
    channel and a few wide channels, as projected keys have."""
    shift = 0.5 * _randn(g, 1, hk, 1, d)
    wide = 1.0 + 2.0 * (torch.rand((1, hk, 1, d), generator=g, device="cuda") > 0.97)
    k = torch.zeros(b, hk, cap, d, dtype=dtype, device="cuda")
    v = torch.zeros(b, hk, cap, d, dtype=dtype, device="cuda")
    k[:, :, :n] = (_randn(g, b, hk, n, d) * wide + shift).to(dtype)
    v[:, :, :n] = _randn(g, b, hk, n, d).to(dtype)
    return k, v


def prepare(case, seed):
    g = _gen(seed)
    b, hq, hk, d = case["b"], case["hq"], case["hk"], case["d"]
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "packed":
        lens = _packed_lengths(case)
        cap = _capacity(max(max(lens), 1))
        total = case["total"]
        s["q"] = _randn(g, total, hq, d, dtype=dt)
        s["k"] = _randn(g, total, hk, d, dtype=dt)
        s["v"] = _randn(g, total, hk, d, dtype=dt)
        s["starts"] = torch.tensor([sum(lens[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
        s["longest"] = max(lens)
        s["k_cache"] = torch.zeros(b, hk, cap, d, dtype=dt, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["desc"] = torch.zeros(b, hk, cap // BLOCK, 2, d, dtype=dt, device="cuda")
        s["out"] = torch.zeros(total, hq, d, dtype=dt, device="cuda")
        return s
    n, cap = case["len"], _capacity(case["len"])
    k, v = _cache(g, b, hk, n, d, dt, cap)
    if case["op"] == "quantize":
        s["k"], s["v"] = k, v
        s["kv4"] = torch.zeros(b, hk, cap // BLOCK, record_bytes(d), dtype=torch.uint8, device="cuda")
        s["k_back"], s["v_back"] = torch.zeros_like(k), torch.zeros_like(v)
        return s
    if case["op"] == "evict":
        s["k"], s["v"] = k, v
        # few keys gather most of the weight, as attention sums do
        s["weights"] = torch.zeros(b, hk, cap, device="cuda")
        s["weights"][:, :, :n] = torch.exp(2.5 * _randn(g, b, hk, n))
        keep = min(n, case["budget"])
        oc = _capacity(case["budget"])
        s["k_out"] = torch.zeros(b, hk, oc, d, dtype=dt, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
        s["desc_out"] = torch.zeros(b, hk, oc // BLOCK, 2, d, dtype=dt, device="cuda")
        s["weights_out"] = torch.zeros(b, hk, oc, device="cuda")
        s["kept"] = torch.zeros(b, hk, case["budget"], dtype=torch.int32, device="cuda")
        s["keep"] = keep
        return s
    s["q"] = _randn(g, b, hq, d, dtype=dt)
    s["out"] = torch.zeros(b, hq, d, dtype=dt, device="cuda")
    s["lse"] = torch.zeros(b, hq, device="cuda")
    lens = _ragged_lengths(case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if case["ragged"] else None
    if case["op"] == "weights":
        s["k"], s["v"] = k, v
        s["weights"] = torch.rand(b, hk, cap, generator=g, device="cuda")
        s["k_new"], s["v_new"] = _randn(g, b, hk, d, dtype=dt), _randn(g, b, hk, d, dtype=dt)
        s["desc"] = _descriptors(k.view(b, hk, cap // BLOCK, BLOCK, d), torch.full((b,), n, device="cuda"))
        return s
    s["kv4"] = torch.cat([_pack(k[i:i + 1], v[i:i + 1]) for i in range(b)])
    m = (n + BLOCK - 1) // BLOCK
    if case["r"] < 1.0:
        ids = torch.rand(b, hk, m, generator=g, device="cuda")
        ids[:, :, m - 1] = 2.0                 # the newest block is always listed
        s["sel"] = ids.topk(_selected(case)).indices.sort().values.to(torch.int32).contiguous()
    return s


# ----------------------------------------------------- the 4-bit cache's format
#
# A group of 64 channels of a token's key or value is held as x = zero + scale * code:
# scale = bf16((max - min) * fp32(1/15)), zero = bf16(min), code = round((x - zero) / scale)
# in 0..15 (0 where the scale is 0), in 32-bit arithmetic, halves to the even code. Sixteen tokens form one record,
#   [key codes][value codes][scales and zeros],
# its codes in the order in which a warp's 32 lanes take them as matrix operands:
#   keys    token 8h + r, channel 64g + 16c + 8j + i:   nibble i of word
#           [g][r][c][2h + j];
#   values  token 8h + 2c + o, channel 64g + 16m + 8e + r: nibble e + 2h + 4o of
#           word [g][r][c][m];
#   scales  token 8h + r, group g: [r][h][g] of {key scale, key zero, value scale,
#           value zero} in bf16.

def record_bytes(d):
    return BLOCK * (d + 8 * (d // GROUP))


def _coded(x):
    """Codes, scale and zero of the groups of the last axis, in 32 bits."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    scale = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).bfloat16()
    zero = lo.bfloat16()
    sf = scale.float().unsqueeze(-1)
    code = torch.where(sf > 0, ((x - zero.float().unsqueeze(-1)) / sf).round().clamp(0, 15), torch.zeros_like(x))
    return code.to(torch.int32).flatten(-2), scale, zero


def _words(nibbles):
    """32-bit words of eight nibbles (last axis, lowest first), in 64-bit integers."""
    at = 4 * torch.arange(8, device=nibbles.device)
    return (nibbles.long() << at).sum(-1)


def _bytes_of(words):
    """Little-endian bytes of 32-bit words held in 64-bit integers."""
    at = 8 * torch.arange(4, device=words.device)
    return ((words.unsqueeze(-1) >> at) & 255).to(torch.uint8)


def _pack(k, v):
    b, h, n, d = k.shape
    m, ng = n // BLOCK, d // GROUP
    kc, ks, kz = _coded(k)
    vc, vs, vz = _coded(v)
    # keys: [h r g c j i] -> [g r c h j] words of i
    kw = _words(kc.view(b, h, m, 2, 8, ng, 4, 2, 8).permute(0, 1, 2, 5, 4, 6, 3, 7, 8))
    # values: [h c o g m e r] -> [g r c m] words of (o h e)
    vw = _words(vc.view(b, h, m, 2, 4, 2, ng, 4, 2, 8).permute(0, 1, 2, 6, 9, 4, 7, 5, 3, 8).flatten(-3))
    meta = torch.stack([ks, kz, vs, vz], -1).view(b, h, m, 2, 8, ng, 4).permute(0, 1, 2, 4, 3, 5, 6)
    meta = meta.contiguous().view(torch.uint8)
    return torch.cat([_bytes_of(kw).flatten(3), _bytes_of(vw).flatten(3), meta.flatten(3)], -1).contiguous()


def _unpack(rec, d):
    """Keys and values [..., tokens, d] that records [..., blocks, bytes] stand for."""
    ng, lead = d // GROUP, rec.shape[:-1]
    code = 512 * ng
    at = 4 * torch.arange(8, device=rec.device, dtype=torch.int32)
    nib = [((rec[..., i * code:(i + 1) * code].contiguous().view(torch.int32).unsqueeze(-1) >> at) & 15) for i in (0, 1)]
    x = len(lead)

    def axes(*p):
        return tuple(range(x)) + tuple(x + i for i in p)

    kc = nib[0].view(*lead, ng, 8, 4, 2, 2, 8).permute(axes(3, 1, 0, 2, 4, 5)).reshape(*lead, BLOCK, d)
    vc = nib[1].view(*lead, ng, 8, 4, 4, 2, 2, 2).permute(axes(5, 2, 4, 0, 3, 6, 1)).reshape(*lead, BLOCK, d)
    meta = rec[..., 2 * code:].contiguous().view(torch.bfloat16).view(*lead, 8, 2, ng, 4)
    meta = meta.permute(axes(1, 0, 2, 3)).reshape(*lead, BLOCK, ng, 1, 4).float()

    def value(codes, s, z):
        return (meta[..., z] + meta[..., s] * codes.view(*lead, BLOCK, ng, GROUP).float()).reshape(*lead[:-1], -1, d)

    return value(kc, 0, 1), value(vc, 2, 3)


# --------------------------------------------------------------- plain forms

def _descriptors(blocks, lens):
    """Per-channel minimum and maximum of the valid keys of each block
    [b, h, m, 16, d]; zeros for blocks with none."""
    b, h, m, _, d = blocks.shape
    pos = torch.arange(m * BLOCK, device=blocks.device).view(1, 1, m, BLOCK, 1)
    ok = pos < lens.view(b, 1, 1, 1, 1)
    lo = blocks.masked_fill(~ok, math.inf).amin(3)
    hi = blocks.masked_fill(~ok, -math.inf).amax(3)
    some = ok[:, :, :, 0]
    return torch.where(some.unsqueeze(3), torch.stack([lo, hi], 3), torch.zeros_like(lo).unsqueeze(3))


def _attend(q, k, v, valid, scale):
    """Attention of one token per row: outputs, log-sum-exp and weights."""
    b, h, n, d = k.shape
    z = torch.matmul(q.float().view(b, h, -1, d), k.transpose(-1, -2)) * scale
    z = z.masked_fill(~valid, -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    w = e / total
    return torch.matmul(w, v).view(b, -1, d), (top + torch.log(total)).view(b, -1), w


def _plain_quantize(s):
    n, d, dt = s["case"]["len"], s["case"]["d"], s["k"].dtype
    s["kv4"].copy_(_pack(s["k"], s["v"]))
    k, v = _unpack(s["kv4"], d)
    s["k_back"][:, :, :n] = k[:, :, :n].to(dt)
    s["v_back"][:, :, :n] = v[:, :, :n].to(dt)
    return {"k": s["k_back"], "v": s["v_back"]}


def _plain_kv4(s):
    c = s["case"]
    b, hk, d, n = c["b"], c["hk"], c["d"], c["len"]
    rec = s["kv4"]
    pos = torch.arange(rec.shape[2] * BLOCK, device="cuda").view(1, 1, -1)
    if "sel" in s:
        ids = s["sel"].long()
        rec = torch.gather(rec, 2, ids.unsqueeze(-1).expand(-1, -1, -1, rec.shape[-1]))
        pos = (ids.unsqueeze(-1) * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(2)
    k, v = _unpack(rec, d)
    lens = s["lens"].view(b, 1, 1) if s["lens"] is not None else n
    out, lse, _ = _attend(s["q"], k, v, (pos < lens).unsqueeze(2), s["scale"])
    s["out"].copy_(out)
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weights(s):
    c = s["case"]
    b, hk, n = c["b"], c["hk"], c["len"]
    lens = s["lens"].long() if s["lens"] is not None else torch.full((b,), n, device="cuda")
    row = torch.arange(b, device="cuda")
    s["k"][row, :, lens - 1] = s["k_new"]
    s["v"][row, :, lens - 1] = s["v_new"]
    j = (lens - 1) // BLOCK
    old, kn = s["desc"][row, :, j], s["k_new"]
    opens = ((lens - 1) % BLOCK == 0).view(b, 1, 1)
    s["desc"][row, :, j] = torch.stack([torch.where(opens, kn, torch.minimum(old[:, :, 0], kn)),
                                        torch.where(opens, kn, torch.maximum(old[:, :, 1], kn))], 2)
    pos = torch.arange(s["k"].shape[2], device="cuda").view(1, 1, -1)
    valid = pos < lens.view(b, 1, 1)
    out, lse, w = _attend(s["q"], s["k"].float(), s["v"].float(), valid.unsqueeze(2), s["scale"])
    total = w.sum(2)
    newest = pos == lens.view(b, 1, 1) - 1
    s["out"].copy_(out)
    s["lse"].copy_(lse)
    # the sum of the token that this step appends begins here
    return {"out": s["out"], "lse": s["lse"], "k": s["k"], "v": s["v"], "desc": s["desc"],
            "weights": s["weights"].copy_(torch.where(valid, torch.where(newest, total, s["weights"] + total),
                                                      s["weights"]))}


def _plain_evict(s):
    c = s["case"]
    n, keep, d = c["len"], s["keep"], c["d"]
    if n > keep:
        old = n - c["recent"]
        order = torch.sort(s["weights"][:, :, :old], dim=-1, descending=True, stable=True).indices
        kept = order[:, :, :keep - c["recent"]].sort().values
        recent = torch.arange(old, n, device="cuda").expand(c["b"], c["hk"], -1)
        kept = torch.cat([kept, recent], -1)
    else:
        kept = torch.arange(n, device="cuda").expand(c["b"], c["hk"], -1)
    rows = kept.unsqueeze(-1).expand(-1, -1, -1, d)
    s["k_out"][:, :, :keep] = torch.gather(s["k"], 2, rows)
    s["v_out"][:, :, :keep] = torch.gather(s["v"], 2, rows)
    s["weights_out"][:, :, :keep] = torch.gather(s["weights"], 2, kept)
    s["kept"].fill_(-1)
    s["kept"][:, :, :keep] = kept.to(torch.int32)
    oc = s["k_out"].shape[2]
    lens = torch.full((c["b"],), keep, device="cuda")
    s["desc_out"].copy_(_descriptors(s["k_out"].view(c["b"], c["hk"], oc // BLOCK, BLOCK, d), lens))
    return {x: s[x] for x in ("k_out", "v_out", "desc_out", "weights_out", "kept")}


def _places(starts, total):
    """Sequence and position of each packed token."""
    at = torch.arange(total, device=starts.device)
    seq = torch.searchsorted(starts.long(), at, right=True) - 1
    return seq, at - starts.long()[seq]


def _causal(q, k, v, seen, scale):
    """One KV head's heads [t, g, d] over its packed keys."""
    z = torch.einsum("tgd,sd->gts", q, k) * scale
    z.masked_fill_(~seen, -math.inf)
    z -= z.amax(-1, keepdim=True)
    z.exp_()
    return torch.einsum("gts,sd->tgd", z, v) / z.sum(-1).t().unsqueeze(-1)


def _plain_packed(s):
    c = s["case"]
    total, hq, hk, d = c["total"], c["hq"], c["hk"], c["d"]
    seq, pos = _places(s["starts"], total)
    seen = (seq.unsqueeze(1) == seq) & (pos.unsqueeze(1) >= pos)
    q, k, v = s["q"].float().view(total, hk, hq // hk, d), s["k"].float(), s["v"].float()
    # (one KV head at a time: the scores of all of them would not fit)
    s["out"].copy_(torch.stack([_causal(q[:, i], k[:, i], v[:, i], seen, s["scale"]) for i in range(hk)], 1)
                   .view(total, hq, d))
    s["k_cache"][seq, :, pos] = s["k"]
    s["v_cache"][seq, :, pos] = s["v"]
    b, _, cap, _ = s["k_cache"].shape
    lens = (s["starts"][1:] - s["starts"][:-1]).long()
    s["desc"].copy_(_descriptors(s["k_cache"].view(b, hk, cap // BLOCK, BLOCK, d), lens))
    return {x: s[x] for x in ("out", "k_cache", "v_cache", "desc")}


# ------------------------------------------------------------ the library's calls

_kept_workspaces = {}


def _workspace(resa, kind, dims, n):
    """The workspace that a program keeps for calls of one shape."""
    key = (kind, dims.batch, dims.n_q_heads, dims.n_kv_heads, dims.head_dim, dims.dtype, dims.max_len, n)
    if key not in _kept_workspaces:
        make = {"weights": resa.alloc_weights_workspace, "kv4": resa.alloc_kv4_workspace,
                "decode": resa.alloc_workspace}[kind]
        _kept_workspaces[key] = make(dims, n)
    return _kept_workspaces[key]


def _own(s):
    import block_sparse_attention_quest_b200 as resa
    c = s["case"]
    op, n = c["op"], c.get("len")
    if op == "quantize":
        resa.kv4_quantize(s["k"], s["v"], n, s["kv4"], c["hq"])
        resa.kv4_dequantize(s["kv4"], n, s["k_back"], s["v_back"], c["hq"])
        return {"k": s["k_back"], "v": s["v_back"]}
    if op == "kv4":
        dims = resa.dims_kv4(s["kv4"], s["q"])
        ws = _workspace(resa, "kv4", dims, n)
        if "sel" in s:
            resa.attend_blocks_kv4(s["q"], s["kv4"], n, s["sel"], s["scale"], s["out"], ws, lse=s["lse"])
        else:
            resa.decode_dense_kv4(s["q"], None, None, s["kv4"], None, n, s["scale"], s["out"], ws,
                                  lse=s["lse"], lens=s["lens"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weights":
        dims = resa.dims_for(s["k"], c["hq"])
        ws = _workspace(resa, "weights", dims, n)
        resa.decode_dense_weights(s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["desc"], s["weights"], n,
                                  s["scale"], s["out"], s["lse"], ws, lens=s["lens"])
        return {x: s[x] for x in ("out", "lse", "k", "v", "desc", "weights")}
    if op == "evict":
        ws = _workspace(resa, "decode", resa.dims_for(s["k"], c["hq"]), n)
        resa.evict(s["k"], s["v"], s["weights"], n, c["budget"], c["recent"], s["k_out"], s["v_out"],
                   s["desc_out"], s["weights_out"], s["kept"], c["hq"], ws)
        return {x: s[x] for x in ("k_out", "v_out", "desc_out", "weights_out", "kept")}
    ws = _workspace(resa, "decode", resa.dims_for(s["k_cache"], c["hq"]), s["k_cache"].shape[2])
    resa.prefill_packed(s["q"], s["k"], s["v"], s["starts"], s["longest"], s["k_cache"], s["v_cache"], s["desc"],
                        s["scale"], s["out"], ws)
    return {x: s[x] for x in ("out", "k_cache", "v_cache", "desc")}


def run(state):
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "kv4": _plain_kv4, "weights": _plain_weights, "evict": _plain_evict,
            "packed": _plain_packed}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what it takes

def work(case):
    b, hq, hk, d = case["b"], case["hq"], case["hk"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "packed":
        lens = _packed_lengths(case)
        pairs = sum(x * (x + 1) // 2 for x in lens)
        blocks = sum((x + BLOCK - 1) // BLOCK for x in lens)
        return {"bytes": case["total"] * d * e * (2 * hq + 4 * hk) + blocks * hk * 2 * d * e,
                "flops": 4 * pairs * hq * d}
    n = case["len"]
    row = hk * d * e                                    # one token's keys, or values
    if op == "quantize":
        rec = b * hk * ((n + BLOCK - 1) // BLOCK) * record_bytes(d)
        return {"bytes": 4 * b * n * row + 2 * rec, "flops": 8 * b * n * hk * d}
    if op == "evict":
        keep = min(n, case["budget"])
        return {"bytes": b * (4 * hk * n + 4 * keep * row + 8 * hk * keep + 2 * (keep + BLOCK - 1) // BLOCK * row),
                "flops": b * hk * (n + 2 * keep * d)}
    lens = _ragged_lengths(case)
    io = 2 * b * hq * d * e + 4 * b * hq
    if op == "weights":
        t = sum(lens)
        return {"bytes": 2 * t * row + 8 * t * hk + io + 6 * b * row, "flops": 4 * t * hq * d}
    t = sum(lens) if case["r"] == 1.0 else b * _selected(case) * BLOCK
    return {"bytes": t * hk * record_bytes(d) // BLOCK + io, "flops": 4 * t * hq * d}


# ------------------------------------------------------------- 64-bit outputs

def _exact_values(rec, d):
    """Records' keys and values in 64 bits: each code looked up by its token
    and channel, as the format's description places it."""
    ng = d // GROUP
    words = rec[..., :1024 * ng].reshape(*rec.shape[:-1], -1, 4).long()
    words = words[..., 0] | words[..., 1] << 8 | words[..., 2] << 16 | words[..., 3] << 24
    meta = rec[..., 1024 * ng:].contiguous().view(torch.bfloat16).double()
    t = torch.arange(BLOCK, device=rec.device).view(-1, 1)
    ch = torch.arange(d, device=rec.device).view(1, -1)
    grp, x = ch // GROUP, ch % GROUP
    k_word = grp * 128 + ((t % 8) * 4 + x // 16) * 4 + (t // 8) * 2 + (x // 8) % 2
    v_word = ng * 128 + grp * 128 + ((x % 8) * 4 + (t % 8) // 2) * 4 + x // 16
    v_nib = (x // 8) % 2 + 2 * (t // 8) + 4 * (t % 2)
    m = (((t % 8) * 2 + t // 8) * ng + grp) * 4
    k = meta[..., m + 1] + meta[..., m] * ((words[..., k_word] >> (4 * (x % 8))) & 15).double()
    v = meta[..., m + 3] + meta[..., m + 2] * ((words[..., v_word] >> (4 * v_nib)) & 15).double()
    return k, v


def _exact_step(q, k, v, n, scale):
    """One row's KV head: heads q [g, d] over keys [n, d], in 64 bits."""
    z = q.double() @ k[:n].t() * scale
    lse = torch.logsumexp(z, -1)
    w = torch.exp(z - lse.unsqueeze(-1))
    return w @ v[:n], lse, w.sum(0)


def exact(case, seed):
    op, b, hq, hk, d = case["op"], case["b"], case["hq"], case["hk"], case["d"]
    g = hq // hk
    s = prepare(case, seed)
    if op == "quantize":
        def back(x):
            y = x.float().unflatten(-1, (-1, GROUP))
            lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
            # which scale, zero and code a value gets is decided in 32 bits, by the format's
            # definition; the value they stand for is then exact
            sc = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device="cuda")).bfloat16().float()
            zo = lo.bfloat16().float()
            code = torch.where(sc > 0, torch.round((y - zo) / sc).clamp(0, 15), torch.zeros_like(y))
            return (zo.double() + sc.double() * code.double()).flatten(-2)
        return {"k": back(s["k"]), "v": back(s["v"])}
    if op == "kv4":
        lens = _ragged_lengths(case)
        out, lse = [], []
        for i in range(b):
            for h in range(hk):
                rec = s["kv4"][i, h]
                n = lens[i]
                if "sel" in s:
                    ids = s["sel"][i, h].long()
                    rec = rec[ids]
                    n = len(ids) * BLOCK - (int(ids[-1]) + 1) * BLOCK + min(n, (int(ids[-1]) + 1) * BLOCK)
                k, v = _exact_values(rec, d)
                o, e, _ = _exact_step(s["q"][i, h * g:(h + 1) * g], k.reshape(-1, d), v.reshape(-1, d), n, s["scale"])
                out.append(o)
                lse.append(e)
        return {"out": torch.stack(out).view(b, hq, d), "lse": torch.stack(lse).view(b, hq)}
    if op == "weights":
        lens = _ragged_lengths(case)
        k, v, w = s["k"], s["v"], s["weights"].double()
        out, lse = [], []
        for i in range(b):
            n = lens[i]
            for h in range(hk):
                k[i, h, n - 1], v[i, h, n - 1] = s["k_new"][i, h], s["v_new"][i, h]
                o, e, x = _exact_step(s["q"][i, h * g:(h + 1) * g], k[i, h].double(), v[i, h].double(), n, s["scale"])
                w[i, h, n - 1] = 0.0
                w[i, h, :n] += x
                out.append(o)
                lse.append(e)
        # what is copied has no other value in 64 bits
        return {"out": torch.stack(out).view(b, hq, d), "lse": torch.stack(lse).view(b, hq), "k": None, "v": None,
                "desc": None, "weights": w}
    if op == "evict":
        return None                                    # copies: nothing is computed
    lens = _packed_lengths(case)
    if sum(x * x for x in lens) * hq * d > 2e12:
        return None
    out = torch.zeros(case["total"], hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for n in lens:
        for h in range(hq):
            q, k, v = (s[x][at:at + n, y].double() for x, y in (("q", h), ("k", h // g), ("v", h // g)))
            z = (q @ k.t() * s["scale"]).masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
            out[at:at + n, h] = torch.softmax(z, -1) @ v
        at += n
    return {"out": out, "k_cache": None, "v_cache": None, "desc": None}
