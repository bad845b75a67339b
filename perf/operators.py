"""The operators of the cached-serving path as they are measured: rotary append, read-back and
shared-prefix attention over the per-(token, head) quantised paged caches.

Every pass is written twice: with ``own`` false as plain torch arithmetic in 32 bits, with ``own``
true as the calls a user makes of ``int4_token_head_kv_gb300``.

append   the step that puts a batch's new tokens into the cache: the position rotation of queries and
         keys, then the cache encoding of keys and values (INT4, INT8 or INT2 rows), and the stored
         rows read back as the values they stand for.
read     cached rows taken out of the cache again (a prefix handed to dense attention, a sequence
         moved between caches).
shared   one decode step of a batch whose sequences start with the same cached prompt: that prompt's
         keys and values are meant to be read once for all of them.
"""
import functools
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 16
DEV = "cuda"

# Lloyd-Max outputs and threshold of the 4-level quantiser of N(0, 1) (J. Max, 1960), as the INT2 rows define them
LM_A, LM_B, LM_T = 0.45278, 1.51042, 0.98160


def _row_bytes(bits, d):
    return d * bits // 8 + 4


def listed():
    append = dict(op="append", bits=4, d=128, dtype="bf16", rot=128, interleaved=False, fused=True, pad=0)
    shared = dict(op="shared", d=128, dtype="bf16", pad=0)
    return [
        # the long-context decode step: 8 sequences, one new token each, positions up to 131072
        dict(append, name="append_decode_8", tokens=8, hq=64, h=8, positions=131072),
        # a decode batch with partly rotated heads in adjacent pairs; a captured batch's padding rows
        dict(append, name="append_decode_33_partial", tokens=33, hq=32, h=8, dtype="fp16", rot=64, interleaved=True,
             pad=1, positions=4096),
        # one prefill chunk of 2048 queries plus the tokens of decoding sequences
        dict(append, name="append_chunk_2109", tokens=2109, hq=32, h=8, positions=32768),
        # the write-throughput batch
        dict(append, name="append_65536", tokens=65536, hq=32, h=8, positions=131072, fused=False),
        # the INT8 cache, small heads, an odd token count
        dict(append, name="append_int8_4097", bits=8, tokens=4097, hq=32, h=4, d=64, rot=64, positions=8192),
        # the INT2 cache
        dict(append, name="append_int2_1000", bits=2, tokens=1000, hq=8, h=2, dtype="fp16", positions=4096, pad=1),
        # a whole batch's rows taken out
        dict(op="read", name="read_int4_65536", bits=4, tokens=65536, h=8, d=128, dtype="bf16", pad=0),
        # one short sequence's rows from the INT8 cache
        dict(op="read", name="read_int8_2047", bits=8, tokens=2047, h=8, d=128, dtype="fp16", pad=1),
        # a few samples of one short prompt
        dict(shared, name="shared_4x512", seqs=4, prefix=512, suffix=64, hq=8, h=2, d=64, dtype="fp16"),
        # the grouped-query decode batch behind a common system prompt, padded to its captured size
        dict(shared, name="shared_32x4096", seqs=32, prefix=4096, suffix=512, hq=32, h=8, pad=1),
        # many questions on one long document
        dict(shared, name="shared_64x32768", seqs=64, prefix=32768, suffix=1024, hq=32, h=8),
        # the long-context heads, a large batch on one very long document
        dict(shared, name="shared_128x131072", seqs=128, prefix=131072, suffix=512, hq=64, h=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "shared", "shared"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    h, g = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 4, 4, 8])
    if op == "append":
        bits = rng.choice([4, 4, 8, 2])
        return dict(op=op, bits=bits, tokens=_log(rng, 1, 32768), hq=h * g, h=h, d=d, dtype=dtype,
                    rot=rng.choice([d, d, d // 2, 16]), interleaved=rng.random() < 0.4, fused=rng.random() < 0.6,
                    positions=_log(rng, 1024, 131072), pad=rng.choice([0, 1]))
    if op == "read":
        return dict(op=op, bits=rng.choice([4, 4, 8, 2]), tokens=_log(rng, 1, 65536), h=h, d=d, dtype=dtype,
                    pad=rng.choice([0, 1]))
    return dict(op=op, seqs=_log(rng, 1, 128), prefix=_log(rng, 64, 65536), suffix=_log(rng, 1, 1024), hq=h * g, h=h,
                d=d, dtype=dtype, pad=rng.choice([0, 0, 1]))


# ------------------------------------------------------------------ plain arithmetic (32 bits)

def _hadamard(d):
    i = torch.arange(d, device=DEV)
    x = i[:, None] & i[None, :]
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    x = x ^ (x >> 1)
    return 1.0 - 2.0 * (x & 1).float()


def _rotate(x, signs):
    """y = H D x / sqrt(d) of vectors in the last dimension."""
    d = x.shape[-1]
    return ((x * signs) @ _hadamard(d)) * (1.0 / math.sqrt(d))


def _unrotate(y, signs):
    d = y.shape[-1]
    return (y @ _hadamard(d)) * (1.0 / math.sqrt(d)) * signs


def _rope(x, cos, sin, rot, interleaved):
    """x [T, heads, d] in 32 bits; cos, sin [T, rot / 2]."""
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((r, x[..., rot:]), dim=-1)


def _encode(x, bits, signs):
    """Rows [..., row bytes] (uint8) of vectors [..., d] in 32 bits."""
    if bits == 8:
        s = (x.abs().amax(-1, keepdim=True) / 127.0).clamp(min=1e-6)
        v = x * (1.0 / s)
        q = torch.trunc(v + torch.where(v >= 0, 0.5, -0.5)).clamp(-128, 127)
        return torch.cat((q.to(torch.int8).view(torch.uint8), s.contiguous().view(torch.uint8)), dim=-1)
    y = _rotate(x, signs)
    if bits == 2:
        s = (y * y).mean(-1, keepdim=True).sqrt().clamp(min=1e-6)
        z = y * (1.0 / s)
        c = (z >= -LM_T).int() + (z >= 0).int() + (z >= LM_T).int()
        b = c[..., 0::4] | (c[..., 1::4] << 2) | (c[..., 2::4] << 4) | (c[..., 3::4] << 6)
        return torch.cat((b.to(torch.uint8), s.contiguous().view(torch.uint8)), dim=-1)
    mn, mx = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    w = ((mx - mn) / 15.0).clamp(min=1e-6).contiguous().view(torch.int32) & -16
    s = w.view(torch.float32)
    zp = torch.round(-mn / s).clamp(0, 15)
    # one rounding of y (1 / s) + zp: the product of two 24-bit numbers is exact in 64 bits
    code = torch.round(y.double() * (1.0 / s).double() + zp.double()).clamp(0, 15).int()
    b = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat((b.to(torch.uint8), (w | zp.int()).view(torch.uint8)), dim=-1)


def _decode(rows, bits, d, signs):
    """The vectors (32 bits) that rows [..., row bytes] stand for."""
    b = rows[..., :d * bits // 8]
    w = rows[..., d * bits // 8:].contiguous()
    if bits == 8:
        return b.contiguous().view(torch.int8).float() * w.view(torch.float32)
    if bits == 2:
        c = torch.stack((b & 3, (b >> 2) & 3, (b >> 4) & 3, b >> 6), dim=-1).flatten(-2)
        lm = torch.tensor([-LM_B, -LM_A, LM_A, LM_B], dtype=torch.float32, device=rows.device)
        return _unrotate(lm[c.long()] * w.view(torch.float32), signs)
    c = torch.stack((b & 15, b >> 4), dim=-1).flatten(-2).float()
    w = w.view(torch.int32)
    return _unrotate((c - (w & 15).float()) * (w & -16).view(torch.float32), signs)


def _plain_append(s):
    rot, inter, bits = s["rot"], s["interleaved"], s["bits"]
    cs = s["cos_sin"][s["positions"]]
    cos, sin = cs[:, :rot // 2], cs[:, rot // 2:]
    q = _rope(s["q"].float(), cos, sin, rot, inter).to(s["q"].dtype)
    live = s["slots"] >= 0
    slots = s["slots"][live]
    k = _rope(s["k"].float(), cos, sin, rot, inter)[live]
    cache = s["cache"]
    cache[slots // BLOCK, 0, slots % BLOCK] = _encode(k, bits, s["signs"])
    cache[slots // BLOCK, 1, slots % BLOCK] = _encode(s["v"].float()[live], bits, s["signs"])
    return (q, *_plain_read(s))


def _plain_read(s):
    slots = s["slots"]
    at = slots.clamp(min=0)
    rows = s["cache"][at // BLOCK, :, at % BLOCK]
    x = _decode(rows, s["bits"], s["d"], s["signs"]) * (slots >= 0)[:, None, None, None]
    x = x.to(s["dtype"])
    return x[:, 0].contiguous(), x[:, 1].contiguous()


def _plain_shared(s):
    d, n, h = s["d"], s["seqs"], s["h"]
    P = s["prefix"] // BLOCK * BLOCK
    rows = s["cache"][s["prefix_blocks"].long()]                       # [blocks, 2, 16, h, row]
    pre = _decode(rows, 4, d, s["signs"])
    kp, vp = (pre[:, i].reshape(P, h, d) for i in (0, 1))
    rest = s["block_tables"][:, P // BLOCK:].long()
    suf = _decode(s["cache"][rest], 4, d, s["signs"])                  # [n, blocks, 2, 16, h, d]
    ks, vs = (suf[:, :, i].reshape(n, -1, h, d) for i in (0, 1))
    q = s["q"].float().reshape(n, h, -1, d) * s["scale"]
    seen = s["seq_lens"].long()
    hide_p = torch.arange(P, device=DEV)[None, :] >= seen[:, None]
    hide_s = torch.arange(ks.shape[1], device=DEV)[None, :] + P >= seen[:, None]
    xp = torch.einsum("nhgd,phd->hngp", q, kp).masked_fill_(hide_p[None, :, None, :], -math.inf)
    xs = torch.einsum("nhgd,nthd->hngt", q, ks).masked_fill_(hide_s[None, :, None, :], -math.inf)
    m = torch.maximum(xp.amax(-1, keepdim=True), xs.amax(-1, keepdim=True)).clamp(min=-1e30)
    xp.sub_(m).exp_()
    xs.sub_(m).exp_()
    total = xp.sum(-1) + xs.sum(-1)
    o = torch.einsum("hngp,phd->nhgd", xp, vp) + torch.einsum("hngt,nthd->nhgd", xs, vs)
    o = o / total.permute(1, 0, 2).clamp(min=1e-30)[..., None]
    return o.reshape(n, -1, d).to(s["q"].dtype)


# ------------------------------------------------------------------ the framework's calls

def _own_append(s):
    import int4_token_head_kv_gb300 as kv
    args = (s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"])
    if s["bits"] == 8:
        q = kv.kv_int8_rope_write(*args, s["cache"], interleaved=s["interleaved"])
    else:
        write = kv.kv_int4_rope_write if s["bits"] == 4 else kv.kv_int2_rope_write
        q = write(*args, s["signs"], s["cache"], interleaved=s["interleaved"])
    return (q, *_own_read(s))


def _own_read(s):
    import int4_token_head_kv_gb300 as kv
    if s["bits"] == 8:
        return kv.kv_int8_read(s["cache"], s["slots"], dtype=s["dtype"])
    read = kv.kv_int4_read if s["bits"] == 4 else kv.kv_int2_read
    return read(s["cache"], s["slots"], s["signs"], dtype=s["dtype"])


def _own_shared(s):
    import int4_token_head_kv_gb300 as kv
    return kv.kv_int4_shared_prefix_attention(s["q"], s["cache"], s["prefix_blocks"], s["prefix"], s["block_tables"],
                                              s["seq_lens"], s["query_start_loc"], s["scale"], s["signs"],
                                              max_seq_len=s["max_seq_len"])


# ------------------------------------------------------------------ what the tools call

def _vectors(gen, tokens, h, d, dtype, outliers):
    x = torch.randn(tokens, h, d, generator=gen, device=DEV)
    if outliers:   # a few strong channels per head, as keys have them
        ch = torch.randint(0, d, (h, 4), generator=gen, device=DEV)
        x = x * torch.ones(h, d, device=DEV).scatter_(1, ch, 10.0)
    return x.to(dtype)


def _random_cache(gen, blocks, bits, h, d, signs):
    rows = [_encode(_vectors(gen, blocks * BLOCK, h, d, torch.bfloat16, k == 0).float(), bits, signs) for k in (0, 1)]
    return torch.stack([r.reshape(blocks, BLOCK, h, -1) for r in rows], dim=1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c, d, h = case, case["d"], case["h"]
    dtype = TYPES[c["dtype"]]
    signs = 1.0 - 2.0 * torch.randint(0, 2, (d,), generator=gen, device=DEV).float()
    if c["op"] == "shared":
        n, P, longest = c["seqs"], c["prefix"], c["prefix"] + c["suffix"]
        shared, mine = P // BLOCK, -(-longest // BLOCK) - P // BLOCK
        cache = _random_cache(gen, shared + n * mine, 4, h, d, signs)
        ids = torch.randperm(shared + n * mine, generator=gen, device=DEV).int()
        prefix_blocks = ids[:shared].contiguous()
        tables = torch.cat((prefix_blocks[None].expand(n, shared), ids[shared:].reshape(n, mine)), dim=1).contiguous()
        lens = P + torch.randint(1, c["suffix"] + 1, (n,), generator=gen, device=DEV).int()
        if c["pad"]:   # the last sequence of a captured batch is a padding row
            lens[-1] = 0
        q = torch.randn(n, c["hq"], d, generator=gen, device=DEV).to(dtype)
        return dict(op="shared", q=q, cache=cache, prefix_blocks=prefix_blocks, prefix=P, block_tables=tables,
                    seq_lens=lens, query_start_loc=torch.arange(n + 1, device=DEV, dtype=torch.int32),
                    scale=d ** -0.5, signs=signs, max_seq_len=longest, seqs=n, d=d, h=h)
    T, bits = c["tokens"], c["bits"]
    blocks = -(-T // BLOCK) + 3
    slots = torch.randperm(blocks * BLOCK, generator=gen, device=DEV)[:T].contiguous()
    if c["pad"]:   # padding tokens of a captured batch
        slots[torch.rand(T, generator=gen, device=DEV) < 0.1] = -1
    if c["op"] == "read":
        cache = _random_cache(gen, blocks, bits, h, d, signs)
        return dict(op="read", cache=cache, slots=slots, signs=signs, bits=bits, d=d, dtype=dtype)
    hq, rot = c["hq"], c["rot"]
    q, k, v = (_vectors(gen, T, n, d, dtype, j == 1) for j, n in enumerate((hq, h, h)))
    if c["fused"]:   # slices of one projection's output, as a layer has them
        q, k, v = torch.cat((q, k, v), dim=1).split((hq, h, h), dim=1)
    positions = torch.randint(0, c["positions"], (T,), generator=gen, device=DEV)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = torch.arange(c["positions"], device=DEV, dtype=torch.float64)[:, None] * inv
    cos_sin = torch.cat((angle.cos(), angle.sin()), dim=1).float()
    cache = torch.zeros(blocks, 2, BLOCK, h, _row_bytes(bits, d), dtype=torch.uint8, device=DEV)
    return dict(op="append", q=q, k=k, v=v, positions=positions, cos_sin=cos_sin, slots=slots, signs=signs, cache=cache,
                rot=rot, interleaved=c["interleaved"], bits=bits, d=d, dtype=dtype)


def run(state):
    if own:
        return {"append": _own_append, "read": _own_read, "shared": _own_shared}[state["op"]](state)
    return {"append": _plain_append, "read": _plain_read, "shared": _plain_shared}[state["op"]](state)


def work(case):
    c, d, h = case, case["d"], case["h"]
    if c["op"] == "shared":
        own_tokens = c["seqs"] * (c["suffix"] + 1) // 2
        keys = c["prefix"] + own_tokens
        rows = c["seqs"] * c["hq"] * d
        return {"bytes": keys * 2 * h * _row_bytes(4, d) + 2 * 2 * rows,
                "flops": 4 * d * c["hq"] * (c["seqs"] * c["prefix"] + own_tokens)}
    T, row = c["tokens"], 2 * h * _row_bytes(c["bits"], d)
    read_back = T * 2 * h * d * 2
    rotations = 2 * T * h * d * (0 if c["bits"] == 8 else d.bit_length() - 1)   # butterflies of one direction
    if c["op"] == "read":
        return {"bytes": T * (row + 8) + read_back, "flops": rotations + 2 * T * h * d * 2}
    return {"bytes": T * (2 * 2 * c["hq"] * d + 2 * 2 * h * d + row + 16 + 4 * c["rot"]) + read_back,
            "flops": 2 * rotations + T * (c["hq"] + h) * c["rot"] * 3 + 2 * T * h * d * 6}


def exact(case, seed):
    """The definitions in 64 bits, on the inputs that prepare() makes."""
    s = prepare(case, seed)
    d, signs = s["d"], s["signs"].double()
    had = functools.reduce(torch.kron, [torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64)] *
                           (d.bit_length() - 1)).to(DEV) / d ** 0.5
    turn = signs[:, None] * had            # x -> x D H / sqrt(d)

    def values(rows, bits):
        n = d * bits // 8
        word = rows[..., n:].contiguous().view(torch.int32)
        if bits == 8:
            return rows[..., :n].contiguous().view(torch.int8).double() * word.view(torch.float32).double()
        per = 8 // bits
        shift = torch.arange(per, device=DEV) * bits
        code = ((rows[..., :n, None].int() >> shift) & ((1 << bits) - 1)).flatten(-2)
        if bits == 2:
            return (code * 2 - 3).sign() * torch.where((code == 1) | (code == 2), LM_A, LM_B).double() @ turn.T * \
                word.view(torch.float32).double()
        scale = torch.bitwise_and(word, ~15).view(torch.float32).double()
        return ((code - torch.bitwise_and(word, 15)).double() * scale) @ turn.T

    if s["op"] == "shared":
        out = []
        P = s["prefix"] // BLOCK * BLOCK
        q, n = s["q"].double(), s["seqs"]
        g = q.shape[1] // s["h"]
        lens = s["seq_lens"].tolist()
        for j in range(s["h"]):
            pre = values(s["cache"][s["prefix_blocks"].long(), :, :, j], 4)
            kp, vp = pre[:, 0].reshape(P, d), pre[:, 1].reshape(P, d)
            all_p = (q[:, j * g:(j + 1) * g].reshape(-1, d) @ kp.T).reshape(n, g, P)
            rows = []
            for b in range(n):
                mine = values(s["cache"][s["block_tables"][b, P // BLOCK:].long(), :, :, j], 4)
                ks, vs = mine[:, 0].reshape(-1, d), mine[:, 1].reshape(-1, d)
                tail, pl = max(lens[b] - P, 0), min(lens[b], P)
                x = torch.cat((all_p[b, :, :pl], q[b, j * g:(j + 1) * g] @ ks[:tail].T), dim=1) * s["scale"]
                if x.shape[1] == 0:
                    rows.append(torch.zeros(g, d, dtype=torch.float64, device=DEV))
                    continue
                w = torch.softmax(x, dim=1)
                rows.append(w[:, :pl] @ vp[:pl] + w[:, pl:] @ vs[:tail])
            out.append(torch.stack(rows))
        return torch.cat(out, dim=1)

    bits, slots = s["bits"], s["slots"]
    if s["op"] == "read":
        at = slots.clamp(min=0)
        x = values(s["cache"][at // BLOCK, :, at % BLOCK], bits) * (slots >= 0)[:, None, None, None]
        return x[:, 0], x[:, 1]

    rot, half = s["rot"], s["rot"] // 2
    table = s["cos_sin"].double()[s["positions"]]
    phase = torch.complex(table[:, :half], table[:, half:])[:, None]

    def turned(x):
        x = x.double()
        first = torch.arange(half, device=DEV) * (2 if s["interleaved"] else 1)
        second = first + (1 if s["interleaved"] else half)
        z = torch.complex(x[..., first], x[..., second]) * phase
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def stored(x):
        """What the encoded vector stands for."""
        if bits == 8:
            step = (x.abs().amax(-1, keepdim=True) / 127).clamp(min=1e-6).float().double()
            return ((x / step).abs() + 0.5).floor().clamp(max=127) * x.sign() * step
        y = x @ turn
        if bits == 2:
            sigma = y.square().mean(-1, keepdim=True).sqrt().clamp(min=1e-6)
            z = y / sigma
            return (torch.where(z >= 0, 1.0, -1.0) * torch.where(((z >= 0) & (z < LM_T)) | ((z < 0) & (z >= -LM_T)), LM_A, LM_B)
                    * sigma) @ turn.T
        low = y.amin(-1, keepdim=True)
        step = ((y.amax(-1, keepdim=True) - low) / 15).clamp(min=1e-6).float().contiguous()
        step = (step.view(torch.int32) // 16 * 16).view(torch.float32).double()
        zero = (-low / step).round().clamp(0, 15)
        return (((y / step + zero).round().clamp(0, 15) - zero) * step) @ turn.T

    live = (slots >= 0)[:, None, None]
    return turned(s["q"]), stored(turned(s["k"])) * live, stored(s["v"].double()) * live
