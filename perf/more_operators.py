"""Rotary writes with several position axes, and attention over key spans, as they are measured: the path of image,
video and packed-prompt tokens through the per-(token, head) quantised paged caches.

Every pass is written twice: with ``own`` false as plain torch arithmetic in 32 bits, with ``own`` true as the calls
a user makes of ``int4_token_head_kv_gb300``.

mrope   a batch's queries and keys rotated by positions on several axes (time, height, width), keys and values
        encoded into the cache (INT4, INT8 or INT2 rows), and the stored rows read back as the values they stand for.
span    attention in which every query row sees the cached keys of a span of its own: its document of a packed prompt,
        a prefix that sees itself whole, an image whose tokens see each other; optionally with capped scores and a
        bias that falls with the distance.  Chunks of queries and single tokens, over the three caches.
"""
import functools
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 16
DEV = "cuda"

# Lloyd-Max outputs and threshold of the 4-level quantiser of N(0, 1) (J. Max, 1960) as the INT2 rows hold them: in fp32
LM_A, LM_B, LM_T = (torch.tensor([v], dtype=torch.float32).item() for v in (0.45278, 1.51042, 0.98160))


def _row_bytes(bits, d):
    return d * bits // 8 + 4


def listed():
    mrope = dict(op="mrope", bits=4, d=128, dtype="bf16", sections="16+24+24", mixed=False, interleaved=False, pad=0)
    span = dict(op="span", bits=4, d=128, dtype="bf16", hq=32, h=8, ragged=False, mask="causal", softcap=0.0, alibi=False,
                pad=0)
    return [
        # the decode step of 8 long conversations with images in them: one new token each
        dict(mrope, name="mrope_decode_8", tokens=8, hq=64, h=8, positions=131072),
        # two images' tokens and the text around them; axes dealt out in turn to the pairs
        dict(mrope, name="mrope_images_2109", tokens=2109, hq=32, h=8, positions=4096, sections="24+20+20", mixed=True),
        # a batch of video prompts
        dict(mrope, name="mrope_video_65536", tokens=65536, hq=32, h=8, positions=32768),
        # images of a small vision tower (two axes, neighbouring pairs) into the INT8 cache, with padding tokens
        dict(mrope, name="mrope_int8_4097", bits=8, tokens=4097, hq=16, h=4, d=64, dtype="fp16", positions=1024,
             sections="16+16", interleaved=True, pad=1),
        # single tokens with capped scores over short INT8 contexts, with padding rows
        dict(span, name="span_decode_int8_16x2048", bits=8, seqs=16, chunk=1, cached=2048, ragged=True, hq=8, h=2, d=64,
             dtype="fp16", softcap=30.0, pad=1),
        # the grouped-query decode batch on packed documents with a distance bias
        dict(span, name="span_decode_32x4096", seqs=32, chunk=1, cached=4096, ragged=True, mask="documents", alibi=True),
        # the long-context heads over the INT2 cache
        dict(span, name="span_decode_int2_8x131072", bits=2, seqs=8, chunk=1, cached=131072, hq=64),
        # drafted tokens checked against their contexts
        dict(span, name="span_draft_16x5", seqs=16, chunk=5, cached=4096, ragged=True, dtype="fp16"),
        # one packed prompt of many documents
        dict(span, name="span_documents_16384", seqs=1, chunk=16384, cached=0, mask="documents"),
        # chunks of 2048 queries over 2048 cached tokens, the first half of each sequence a prefix that sees itself whole
        dict(span, name="span_prefix_4x2048", seqs=4, chunk=2048, cached=2048, mask="prefix", softcap=50.0),
        # prompts with images in them over the INT8 cache, odd lengths, padding rows
        dict(span, name="span_images_int8_3x4099", bits=8, seqs=3, chunk=4099, cached=0, ragged=True, mask="images", hq=16,
             h=2, pad=1),
        # a late chunk of a long prompt
        dict(span, name="span_chunk_2048_at_32768", seqs=1, chunk=2048, cached=32768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:   # no more than the largest listed ones
            return c


def _draw(rng):
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    h, g = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 4, 4, 8])
    bits = rng.choice([4, 4, 8, 2])
    if rng.random() < 0.4:
        pairs = rng.choice([d, d, d // 2]) // 2
        axes = rng.choice([2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = "+".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))
        return dict(op="mrope", bits=bits, tokens=_log(rng, 1, 32768), hq=h * g, h=h, d=d, dtype=dtype, sections=sections,
                    mixed=rng.random() < 0.4, interleaved=rng.random() < 0.4, positions=_log(rng, 256, 131072),
                    pad=rng.choice([0, 1]))
    kind = rng.choice(["decode", "draft", "chunk", "chunk"])
    if kind == "decode":
        seqs, chunk, cached = _log(rng, 1, 64), 1, _log(rng, 1, 32768)
    elif kind == "draft":
        seqs, chunk, cached = _log(rng, 1, 32), rng.randint(2, 17), _log(rng, 1, 16384)
    else:
        seqs, chunk, cached = rng.randint(1, 4), _log(rng, 18, 4100), rng.choice([0, _log(rng, 1, 8192)])
    return dict(op="span", bits=bits, seqs=seqs, chunk=chunk, cached=cached, ragged=rng.random() < 0.6, hq=h * g, h=h, d=d,
                dtype=dtype, mask=rng.choice(["causal", "documents", "prefix", "images"]),
                softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.3, pad=rng.choice([0, 0, 1]))


# ------------------------------------------------------------------ a span case's batch (the same for every seed)

@functools.lru_cache(maxsize=64)
def _batch_of(key):
    """Per sequence (tokens, the last of them queries), and per query row its span (begin, end): host integers."""
    seqs, chunk, cached, ragged, mask, pad = key
    rng = random.Random(repr(key))
    shapes, begin, end = [], [], []
    for i in range(seqs):
        q = rng.randint(max(1, chunk // 2), chunk) if ragged else chunk
        c = rng.randint(cached // 8, cached) if ragged else cached
        if pad and i == seqs - 1 and seqs > 1:   # a padding row of a captured batch: one query, no tokens
            shapes.append((0, 1))
            begin.append(0)
            end.append(0)
            continue
        total = c + q
        shapes.append((total, q))
        # documents (or images and the text between them), some short, some long
        starts = [0]
        while starts[-1] < total:
            starts.append(starts[-1] + _log(rng, max(1, total // 64), max(2, total // 4)))
        prefix = rng.randint(total // 4, total // 2)
        doc = 0
        for pos in range(c, total):
            while starts[doc + 1] <= pos:
                doc += 1
            b, e = 0, pos + 1
            if mask == "documents":
                b = starts[doc]
            elif mask == "prefix":
                e = max(e, prefix)
            elif mask == "images":   # every second stretch is an image; pairs of stretches are documents
                b = starts[doc - doc % 2]
                if doc % 2:
                    e = min(starts[doc + 1], total)
            if pad and rng.random() < 0.02:   # a row that sees nothing
                b = e
            begin.append(b)
            end.append(e)
    return shapes, begin, end


def _batch(c):
    return _batch_of((c["seqs"], c["chunk"], c["cached"], c["ragged"], c["mask"], c["pad"]))


# ------------------------------------------------------------------ plain arithmetic (32 bits)

def _butterflies(x):
    """The Walsh-Hadamard transform of vectors in the last dimension, strides 1, 2, 4, ... as the rows define it."""
    d = x.shape[-1]
    h = 1
    while h < d:
        y = x.reshape(*x.shape[:-1], d // (2 * h), 2, h)
        a, b = y[..., 0, :], y[..., 1, :]
        x = torch.stack((a + b, a - b), dim=-2).reshape(x.shape)
        h *= 2
    return x


def _rotate(x, signs):
    """y = H D x / sqrt(d) of vectors in the last dimension."""
    return _butterflies(x * signs) * (1.0 / math.sqrt(x.shape[-1]))


def _unrotate(y, signs):
    return _butterflies(y) * (1.0 / math.sqrt(y.shape[-1])) * signs


def _rope(x, cos, sin, interleaved):
    """x [T, heads, d] in 32 bits; cos, sin [T, pairs]."""
    rot = 2 * cos.shape[-1]
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((r, x[..., rot:]), dim=-1)


def _sections(case):
    """Pairs of each axis."""
    return tuple(int(n) for n in case["sections"].split("+"))


def _pair_axes(sections, mixed):
    """The axis of every pair: the sections one after another, or dealt out in turn while they last."""
    if not mixed:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while len(out) < sum(sections):
        for a in range(len(sections)):
            if left[a] > 0:
                left[a] -= 1
                out.append(a)
    return out


def _encode(x, bits, signs):
    """Rows [..., row bytes] (uint8) of vectors [..., d] in 32 bits."""
    if bits == 8:
        s = (x.abs().amax(-1, keepdim=True) / 127.0).clamp(min=1e-6)
        v = x * (1.0 / s)
        q = torch.trunc(v + torch.where(v >= 0, 0.5, -0.5)).clamp(-128, 127)
        return torch.cat((q.to(torch.int8).view(torch.uint8), s.contiguous().view(torch.uint8)), dim=-1)
    y = _rotate(x, signs)
    if bits == 2:
        a = y * y   # the squares folded in halves
        while a.shape[-1] > 1:
            a = a[..., :a.shape[-1] // 2] + a[..., a.shape[-1] // 2:]
        s = (a / y.shape[-1]).sqrt().clamp(min=1e-6)
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


def _read_rows(s):
    slots = s["slots"]
    at = slots.clamp(min=0)
    rows = s["cache"][at // BLOCK, :, at % BLOCK]
    x = _decode(rows, s["bits"], s["d"], s["signs"]) * (slots >= 0)[:, None, None, None]
    x = x.to(s["q"].dtype)
    return x[:, 0].contiguous(), x[:, 1].contiguous()


def _plain_mrope(s):
    axes = torch.tensor(_pair_axes(s["sections"], s["mixed"]), device=DEV)
    n = len(axes)
    pair = torch.arange(n, device=DEV)
    at = s["positions"][axes].T                                        # [T, pairs]
    cos, sin = s["cos_sin"][at, pair], s["cos_sin"][at, n + pair]
    q = _rope(s["q"].float(), cos, sin, s["interleaved"]).to(s["q"].dtype)
    live = s["slots"] >= 0
    slots = s["slots"][live]
    k = _rope(s["k"].float(), cos, sin, s["interleaved"])[live]
    cache = s["cache"]
    cache[slots // BLOCK, 0, slots % BLOCK] = _encode(k, s["bits"], s["signs"])
    cache[slots // BLOCK, 1, slots % BLOCK] = _encode(s["v"].float()[live], s["bits"], s["signs"])
    return (q, *_read_rows(s))


def _softmax_rows(x, seen, keys_of):
    """Weights of logits x over the visible keys (in place): rows that see none have only zeros."""
    x.masked_fill_(~seen, -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    return keys_of(x) / total.clamp(min=1e-30)


def _bias(x, s, pos, keys, slopes):
    """Capped scores and the distance bias on logits x (in place)."""
    if s["softcap"] > 0.0:
        x.div_(s["softcap"]).tanh_().mul_(s["softcap"])
    if slopes is not None:
        x.sub_(slopes * (pos - keys).abs().float())


def _plain_span(s):
    d, h = s["d"], s["h"]
    out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    g = s["q"].shape[1] // h
    if s["chunk"] == 1:   # single tokens: the batch at once
        n, width = s["seq_lens"].shape[0], s["block_tables"].shape[1] * BLOCK
        keys = torch.arange(width, device=DEV)
        begin = s["key_begin"] if s["key_begin"] is not None else torch.zeros_like(s["seq_lens"])
        end = s["key_end"] if s["key_end"] is not None else s["seq_lens"]
        seen = (keys >= begin[:, None]) & (keys < torch.minimum(end, s["seq_lens"])[:, None])
        slopes = s["alibi"].reshape(h, g)[:, None, :, None] if s["alibi"] is not None else None
        rows = s["cache"][s["block_tables"].long()]                    # [n, blocks, 2, 16, h, row]
        kx, vx = (_decode(rows[:, :, i], s["bits"], d, s["signs"]).reshape(n, width, h, d) for i in (0, 1))
        x = torch.einsum("nhgd,nthd->hngt", s["q"].float().reshape(n, h, g, d) * s["scale"], kx)
        _bias(x, s, (s["seq_lens"] - 1)[None, :, None, None], keys, slopes)
        o = _softmax_rows(x, seen[None, :, None, :], lambda w: torch.einsum("hngt,nthd->hngd", w, vx))
        return o.permute(1, 0, 2, 3).reshape(n, -1, d).to(out.dtype)
    slopes = s["alibi"].reshape(h, g)[:, :, None, None] if s["alibi"] is not None else None
    row = 0
    for i, (total, m) in enumerate(s["shapes"]):
        row += m
        if total == 0:   # a padding row
            out[row - m:row] = 0
            continue
        blocks = s["block_tables"][i, :-(-total // BLOCK)].long()
        rows = s["cache"][blocks]
        kx, vx = (_decode(rows[:, j], s["bits"], d, s["signs"]).reshape(-1, h, d)[:total] for j in (0, 1))
        keys = torch.arange(total, device=DEV)
        step = max(1, 2 ** 31 // (h * g * total))                      # rows whose logits fit 8 GB
        for r in range(0, m, step):
            n = min(step, m - r)
            at = slice(row - m + r, row - m + r + n)
            pos = torch.arange(total - m + r, total - m + r + n, device=DEV)[:, None]
            begin = s["key_begin"][at, None] if s["key_begin"] is not None else 0
            end = s["key_end"][at, None] if s["key_end"] is not None else pos + 1
            x = torch.einsum("mhgd,thd->hgmt", s["q"][at].float().reshape(n, h, g, d) * s["scale"], kx)
            _bias(x, s, pos, keys, slopes)
            o = _softmax_rows(x, (keys >= begin) & (keys < end), lambda w: torch.einsum("hgmt,thd->hgmd", w, vx))
            out[at] = o.permute(2, 0, 1, 3).reshape(n, -1, d).to(out.dtype)
    return out


# ------------------------------------------------------------------ the framework's calls

def _own_mrope(s):
    import int4_token_head_kv_gb300 as kv
    write = {4: kv.kv_int4_mrope_write, 8: kv.kv_int8_mrope_write, 2: kv.kv_int2_mrope_write}[s["bits"]]
    read = {4: kv.kv_int4_read, 8: kv.kv_int8_read, 2: kv.kv_int2_read}[s["bits"]]
    signs = () if s["bits"] == 8 else (s["signs"],)
    q = write(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["sections"], s["slots"], *signs, s["cache"],
              interleaved=s["interleaved"], mixed_sections=s["mixed"])
    return (q, *read(s["cache"], s["slots"], *signs, dtype=s["q"].dtype))


def _own_span(s):
    import int4_token_head_kv_gb300 as kv
    attend = {4: kv.kv_int4_span_attention, 8: kv.kv_int8_span_attention, 2: kv.kv_int2_span_attention}[s["bits"]]
    signs = () if s["bits"] == 8 else (s["signs"],)
    return attend(s["q"], s["cache"], s["block_tables"], s["seq_lens"], s["query_start_loc"], s["scale"], *signs,
                  max_query_len=s["max_query_len"], max_seq_len=s["max_seq_len"], key_begin=s["key_begin"],
                  key_end=s["key_end"], softcap=s["softcap"], alibi_slopes=s["alibi"])


# ------------------------------------------------------------------ what the tools call

def _vectors(gen, tokens, h, d, dtype, outliers):
    x = torch.randn(tokens, h, d, generator=gen, device=DEV)
    if outliers:   # a few strong channels per head, as keys have them
        ch = torch.randint(0, d, (h, 4), generator=gen, device=DEV)
        x = x * torch.ones(h, d, device=DEV).scatter_(1, ch, 10.0)
    return x.to(dtype)


def _random_cache(gen, blocks, bits, h, d, signs):
    cache = torch.empty(blocks, 2, BLOCK, h, _row_bytes(bits, d), dtype=torch.uint8, device=DEV)
    for b in range(0, blocks, 8192):
        n = min(8192, blocks - b)
        for i in (0, 1):
            x = _vectors(gen, n * BLOCK, h, d, torch.bfloat16, i == 0).float()
            cache[b:b + n, i] = _encode(x, bits, signs).reshape(n, BLOCK, h, -1)
    return cache


def _prepare_span(c, gen, signs):
    d, h, bits = c["d"], c["h"], c["bits"]
    shapes, begin, end = _batch(c)
    lens = [n for n, _ in shapes]
    width = max(1, max(-(-n // BLOCK) for n in lens))
    blocks = sum(-(-n // BLOCK) for n in lens) + 3
    cache = _random_cache(gen, blocks, bits, h, d, signs)
    ids = torch.randperm(blocks, generator=gen, device=DEV).int()
    tables = torch.zeros(len(lens), width, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(lens):
        n = -(-n // BLOCK)
        tables[i, :n] = ids[at:at + n]
        at += n
    starts = [0]
    for _, m in shapes:
        starts.append(starts[-1] + m)
    q = torch.randn(starts[-1], c["hq"], d, generator=gen, device=DEV).to(TYPES[c["dtype"]])
    # what the mask needs: documents begin, prefixes and images end, and rows that see nothing need both
    need_begin, need_end = c["mask"] in ("documents", "images"), c["mask"] in ("prefix", "images")
    if c["pad"]:
        need_begin = need_end = True
    ints = functools.partial(torch.tensor, dtype=torch.int32, device=DEV)
    slopes = 2.0 ** (-8.0 * (torch.arange(c["hq"], device=DEV, dtype=torch.float32) + 1.0) / c["hq"])
    return dict(op="span", q=q, cache=cache, block_tables=tables, seq_lens=ints(lens), query_start_loc=ints(starts),
                key_begin=ints(begin) if need_begin else None, key_end=ints(end) if need_end else None, scale=d ** -0.5,
                signs=signs, softcap=c["softcap"], alibi=slopes if c["alibi"] else None, shapes=shapes, chunk=c["chunk"],
                max_query_len=max(m for _, m in shapes), max_seq_len=max(lens), bits=bits, d=d, h=h)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c, d, h, bits = case, case["d"], case["h"], case["bits"]
    signs = 1.0 - 2.0 * torch.randint(0, 2, (d,), generator=gen, device=DEV).float()
    if c["op"] == "span":
        return _prepare_span(c, gen, signs)
    sections = _sections(c)
    T, rot = c["tokens"], 2 * sum(sections)
    blocks = -(-T // BLOCK) + 3
    slots = torch.randperm(blocks * BLOCK, generator=gen, device=DEV)[:T].contiguous()
    if c["pad"]:   # padding tokens of a captured batch
        slots[torch.rand(T, generator=gen, device=DEV) < 0.1] = -1
    # slices of one projection's output, as a layer has them
    x = [_vectors(gen, T, n, d, TYPES[c["dtype"]], j == 1) for j, n in enumerate((c["hq"], h, h))]
    q, k, v = torch.cat(x, dim=1).split((c["hq"], h, h), dim=1)
    # frames, rows and columns of images and videos: each axis has its own position
    positions = torch.randint(0, c["positions"], (len(sections), T), generator=gen, device=DEV)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    angle = torch.arange(c["positions"], device=DEV, dtype=torch.float64)[:, None] * inv
    cos_sin = torch.cat((angle.cos(), angle.sin()), dim=1).float()
    cache = torch.zeros(blocks, 2, BLOCK, h, _row_bytes(bits, d), dtype=torch.uint8, device=DEV)
    return dict(op="mrope", q=q, k=k, v=v, positions=positions, cos_sin=cos_sin, slots=slots, signs=signs, cache=cache,
                sections=sections, mixed=c["mixed"], interleaved=c["interleaved"], bits=bits, d=d)


def run(state):
    if own:
        return {"mrope": _own_mrope, "span": _own_span}[state["op"]](state)
    return {"mrope": _plain_mrope, "span": _plain_span}[state["op"]](state)


def work(case):
    c, d, h = case, case["d"], case["h"]
    if c["op"] == "mrope":
        T, row, rot, axes = c["tokens"], 2 * h * _row_bytes(c["bits"], d), 2 * sum(_sections(c)), len(_sections(c))
        rotations = 2 * T * h * d * (0 if c["bits"] == 8 else d.bit_length() - 1)   # butterflies of one direction
        return {"bytes": T * (2 * 2 * c["hq"] * d + 2 * 2 * h * d + row + 8 + 8 * axes + 4 * rot + 2 * h * d * 2),
                "flops": 2 * rotations + T * (c["hq"] + h) * rot * 3 + 2 * T * h * d * 6}
    shapes, begin, end = _batch(c)
    pairs = rows = keys = 0
    for _, m in shapes:   # visible pairs, and the keys that some row of the sequence sees
        spans = sorted((b, e) for b, e in zip(begin[rows:rows + m], end[rows:rows + m]) if e > b)
        rows += m
        pairs += sum(e - b for b, e in spans)
        upto = 0
        for b, e in spans:
            keys += max(0, e - max(b, upto))
            upto = max(upto, e)
    return {"bytes": keys * 2 * h * _row_bytes(c["bits"], d) + 2 * 2 * rows * c["hq"] * d, "flops": 4 * d * c["hq"] * pairs}


def exact(case, seed):
    """The definitions in 64 bits, on the inputs that prepare() makes."""
    if case["op"] == "span" and work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    d, signs, bits = s["d"], s["signs"].double(), s["bits"]
    had = functools.reduce(torch.kron, [torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64)] *
                           (d.bit_length() - 1)).to(DEV) / d ** 0.5
    turn = signs[:, None] * had            # x -> x D H / sqrt(d)

    def values(rows):
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

    if s["op"] == "span":
        shapes, begin, end = _batch(case)
        g = s["q"].shape[1] // s["h"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        row = 0
        for i, (total, m) in enumerate(shapes):
            # rows in stretches, each against the keys that one of its rows sees
            step = max(1, min(m, 256))
            for r in range(0, m, step):
                rows = range(row + r, row + min(m, r + step))
                live = [(begin[j], end[j]) for j in rows if end[j] > begin[j]]
                if not live:
                    continue
                lo, hi = min(b for b, _ in live) // BLOCK * BLOCK, max(e for _, e in live)
                cached = s["cache"][s["block_tables"][i, lo // BLOCK:-(-hi // BLOCK)].long()]
                key = torch.arange(lo, hi, device=DEV, dtype=torch.float64)
                pos = torch.tensor([total - m + j - row for j in rows], device=DEV, dtype=torch.float64)
                hide = torch.tensor([[begin[j], max(begin[j], end[j])] for j in rows], device=DEV, dtype=torch.float64)
                hide = (key < hide[:, :1]) | (key >= hide[:, 1:])
                for j in range(s["h"]):
                    both = values(cached[:, :, :, j])
                    kx, vx = (both[:, n].reshape(-1, d)[:hi - lo] for n in (0, 1))
                    for u in range(j * g, j * g + g):
                        x = s["q"][rows.start:rows.stop, u].double() @ kx.T * s["scale"]
                        if s["softcap"] > 0:
                            x = s["softcap"] * torch.tanh(x / s["softcap"])
                        if s["alibi"] is not None:
                            x = x - s["alibi"][u].double() * (pos[:, None] - key).abs()
                        w = torch.softmax(x.masked_fill(hide, -math.inf), dim=1).nan_to_num(nan=0.0)
                        out[rows.start:rows.stop, u] = w @ vx
            row += m
        return out

    axes = torch.tensor(_pair_axes(s["sections"], s["mixed"]), device=DEV)
    half = axes.numel()
    pair = torch.arange(half, device=DEV)
    at = s["positions"].T[:, axes]
    phase = torch.complex(s["cos_sin"].double()[at, pair], s["cos_sin"].double()[at, half + pair])[:, None]

    def turned(x):
        x = x.double()
        first = pair * (2 if s["interleaved"] else 1)
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

    live = (s["slots"] >= 0)[:, None, None]
    return turned(s["q"]), stored(turned(s["k"])) * live, stored(s["v"].double()) * live
