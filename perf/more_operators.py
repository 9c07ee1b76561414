"""Operators over quantized caches, as they are measured: each in a plain form of elementary torch
operations, and as the calls that a user makes of the library.

  cross   attention of query rows to every cached key of their sequence (an encoder's states)
  prefix  a decode step's attention of sequences that share a prefix, the prefix held once
  append  new rows encoded into the cache as they come, and read back as values
  read    cached rows read back as values

Both sides take the same cache bytes.  What a cache holds in fewer than 16 bits is returned as the
values that it stands for.
"""
import math

import numpy as np
import torch

own = False

D = 128
F16, Q8_0, Q4_0, TURBO4 = 0, 1, 2, 3
ROW = {F16: 256, Q8_0: 136, Q4_0: 72, TURBO4: 66}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
SCALE = 1 / math.sqrt(D)


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a short system prompt before sixteen chats that have hardly begun: launch latency
        dict(name="16 chats behind 4096 shared tokens", op="prefix", seqs=16, groups=1, prefix=4096, past=255,
             n_q=8, n_kv=2, pk=Q8_0, pv=Q8_0, k=Q8_0, v=Q8_0, paged=False),
        # many users ask about one long document
        dict(name="64 chats behind 32768 shared tokens", op="prefix", seqs=64, groups=1, prefix=32768, past=511,
             n_q=32, n_kv=8, pk=Q4_0, pv=Q4_0, k=Q4_0, v=Q4_0, paged=False),
        # three prompts of uneven lengths and shares under the asymmetric contract, in pages
        dict(name="24 chats behind three prompts", op="prefix", seqs=24, groups=3, prefix=16411, past=701,
             n_q=40, n_kv=8, pk=F16, pv=Q8_0, k=F16, v=Q8_0, paged=True),
        # a batch of continuations of one full slot
        dict(name="128 continuations of 200704 tokens", op="prefix", seqs=128, groups=1, prefix=200704, past=1023,
             n_q=32, n_kv=4, pk=Q8_0, pv=Q8_0, k=F16, v=F16, paged=False),
        # one decoder token for each of sixteen inputs
        dict(name="single tokens over 1500 states", op="cross", seqs=16, rows=16, keys=1500, n_q=8, n_kv=2,
             k=F16, v=F16, type="f16", paged=False),
        # five beams for each of 24 inputs of uneven lengths, in pages
        dict(name="beams over up to 4096 states", op="cross", seqs=24, rows=120, keys=4096, n_q=40, n_kv=8,
             k=F16, v=Q8_0, type="f16", paged=True),
        # whole targets scored against their inputs, bf16 projections
        dict(name="3011 target rows over 1500 states", op="cross", seqs=8, rows=3011, keys=1500, n_q=32, n_kv=8,
             k=Q8_0, v=Q8_0, type="bf16", paged=False),
        # an ubatch of questions against one long input
        dict(name="2048 rows over 32768 states", op="cross", seqs=1, rows=2048, keys=32768, n_q=32, n_kv=8,
             k=Q8_0, v=Q4_0, type="f16", paged=False),
        # the states of eight inputs, views of a fused bf16 projection, into empty caches
        dict(name="append the states of eight inputs", op="append", seqs=8, rows=9001, past=0, n_kv=8, k=F16, v=Q8_0,
             type="bf16", paged=False, update=True),
        # one token each for sixteen slots, kept in four bits
        dict(name="append 16 single tokens", op="append", seqs=16, rows=16, past=2047, n_kv=8, k=TURBO4, v=TURBO4,
             type="bf16", paged=True, update=True),
        # two long slots read back whole, to be stored or moved
        dict(name="read 98304 tokens of two slots", op="read", seqs=2, rows=98304, past=65536, n_kv=8, k=Q4_0, v=Q4_0,
             type="f16", paged=False),
        # the last tokens of sixteen short slots in pages, as fp32
        dict(name="read 5003 tokens of 16 slots", op="read", seqs=16, rows=5003, past=4097, n_kv=8, k=Q8_0, v=TURBO4,
             type="f32", paged=True),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _draw(rng):
    op = rng.choice(["prefix", "cross", "append", "read"])
    n_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 5, 8])
    codec = lambda: rng.choice([F16, Q8_0, Q4_0, TURBO4])
    case = dict(op=op, n_kv=n_kv, k=codec(), v=codec(), paged=rng.random() < 0.5)
    if op == "prefix":
        seqs = _log(rng, 1, 128)
        return dict(case, seqs=seqs, groups=rng.randint(1, min(seqs, 4)), prefix=_log(rng, 1, 200704),
                    past=_log(rng, 1, 2048), n_q=n_kv * group, pk=codec(), pv=codec())
    seqs = _log(rng, 1, 24)
    if op == "cross":
        return dict(case, seqs=seqs, rows=_log(rng, seqs, 4096), keys=_log(rng, 1, 65536), n_q=n_kv * group,
                    type=rng.choice(["f16", "bf16"]))
    kind = rng.choice(["f16", "bf16", "f32"])
    if op == "append":
        return dict(case, seqs=seqs, rows=_log(rng, seqs, 16384), past=rng.choice([0, rng.randint(1, 2048)]),
                    type=kind, update=rng.random() < 0.5)
    past = _log(rng, 1, 65536)
    case = dict(case, seqs=min(seqs, past), past=past, type=kind)
    most = sum(lengths(case))
    return dict(case, rows=_log(rng, 1, min(most, 98304)))


def draw(rng):
    most = [max(work(c)[u] for c in listed()) for u in ("bytes", "flops")]
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return case


def lengths(case):
    """Cached tokens per sequence: the longest first, the rest spread below it."""
    n, longest = case["seqs"], case["keys"] if case["op"] == "cross" else case["past"]
    return [max(longest * (n - s) // n, 0 if case["op"] == "append" else 1) for s in range(n)]


def shares(total, parts):
    """A total in uneven whole parts of at least one each."""
    weights = [2 + (7 * i) % 5 for i in range(parts)]
    rest = total - parts
    got = [1 + rest * w // sum(weights) for w in weights]
    got[0] += total - sum(got)
    return got


def prefixes(case):
    return [max(1, case["prefix"] * (case["groups"] - g) // case["groups"]) for g in range(case["groups"])]


def counts(case):
    """Rows per sequence."""
    if case["op"] != "read":
        return shares(case["rows"], case["seqs"])
    lens = lengths(case)  # a part of what each has cached, the rest from the first that has more
    got = [case["rows"] * n // sum(lens) for n in lens]
    for i, n in enumerate(lens):
        got[i] += min(n - got[i], case["rows"] - sum(got))
    return got


def work(case):
    row = case["n_kv"] * (ROW[case["k"]] + ROW[case["v"]])
    if case["op"] == "prefix":
        n_q, keys, size = case["n_q"], prefixes(case), shares(case["seqs"], case["groups"])
        own_keys = sum(lengths(case))
        shared = sum(keys) * case["n_kv"] * (ROW[case["pk"]] + ROW[case["pv"]])
        seen = own_keys + sum(a * b for a, b in zip(keys, size))
        return {"bytes": shared + own_keys * row + case["seqs"] * n_q * 512, "flops": 4 * D * n_q * seen}
    if case["op"] == "cross":
        n_q = case["n_q"]
        seen = sum(a * b for a, b in zip(lengths(case), counts(case)))
        return {"bytes": sum(lengths(case)) * row + case["rows"] * n_q * 512, "flops": 4 * D * n_q * seen}
    values = 2 * sum(counts(case)) * case["n_kv"] * D
    # an append's codes are written, and read back
    codes = sum(counts(case)) * row * (2 if case["op"] == "append" else 1)
    return {"bytes": codes + values * SIZE[case["type"]] * (2 if case["op"] == "append" else 1), "flops": values}


# ------------------------------------------------------------------------------------- cache layout

def unit_offsets(codec, side):
    """[16][row bytes]: where byte cb of row r lies inside a 16-token unit of the cache."""
    r, cb = np.arange(16)[:, None], np.arange(ROW[codec])[None, :]
    g, rh, tig, par = r & 7, r >> 3, (r & 7) >> 1, r & 1
    if codec == F16:
        d, k = cb >> 1, cb & 1
        if side == 0:
            return (2 * (d >> 5) + rh) * 512 + (4 * g + ((d >> 2) & 3)) * 16 + ((d >> 4) & 1) * 8 + (d & 3) * 2 + k
        return (d >> 4) * 512 + (4 * ((d & 15) >> 1) + tig) * 16 + (rh * 4 + (d & 1) * 2 + par) * 2 + k
    if codec == Q8_0:
        b, x = cb // 34, cb % 34
        e = x - 2
        if side == 0:
            q = b * 512 + (4 * g + ((e >> 2) & 3)) * 16 + (2 * rh + (e >> 4)) * 4 + (e & 3)
            return np.where(x < 2, 2048 + g * 16 + rh * 8 + b * 2 + x, q)
        q = b * 512 + (4 * ((e & 15) >> 1) + tig) * 16 + ((e >> 4) * 2 + rh) * 4 + par * 2 + (e & 1)
        return np.where(x < 2, 2048 + tig * 32 + b * 8 + rh * 4 + par * 2 + x, q)
    if codec == Q4_0:
        b, x = cb // 18, cb % 18
        is_scale, k_scale, v_scale = x < 2, 1024 + g * 16 + rh * 8 + b * 2 + x, 1024 + tig * 32 + b * 8 + rh * 4 + par * 2 + x
        j = x - 2
    else:
        b, j = (cb - 2) // 16, (cb - 2) % 16
        is_scale, k_scale, v_scale = cb < 2, 1024 + g * 4 + rh * 2 + cb, 1024 + tig * 8 + rh * 4 + par * 2 + cb
    if side == 0:
        return np.where(is_scale, k_scale, (b >> 1) * 512 + (4 * g + (j >> 2)) * 16 + ((b & 1) * 2 + rh) * 4 + (j & 3))
    mt = 2 * b + (j >> 3)
    return np.where(is_scale, v_scale, (mt >> 2) * 512 + (4 * (j & 7) + tig) * 16 + (mt & 3) * 4 + par * 2 + rh)


_OFFSETS = {}


def offsets(codec, side):
    if (codec, side) not in _OFFSETS:
        _OFFSETS[codec, side] = torch.from_numpy(np.ascontiguousarray(unit_offsets(codec, side))).cuda()
    return _OFFSETS[codec, side]


def units(seq, head, pos, n_kv, capacity, table):
    """The unit that holds token `pos` of (seq, kv head), in the cache or the page pool."""
    if table is None:
        return (seq * n_kv + head) * (capacity // 16) + pos // 16
    return (table[seq, pos // 256].long() * n_kv + head) * 16 + (pos // 16) % 16


def row_bytes_at(cache, codec, side, unit, row):
    """Canonical bytes of rows (unit, row), each of any one shape."""
    return cache[unit[..., None] * (16 * ROW[codec]) + offsets(codec, side)[row]]


# ------------------------------------------------------------------------------------- codecs

def _splitmix_sign(n):
    z = (0x4B5651 + 0x9E3779B97F4A7C15 * (n + 1)) & (2**64 - 1)
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & (2**64 - 1)
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & (2**64 - 1)
    return -1.0 if ((z ^ (z >> 31)) >> 63) & 1 else 1.0


SIGNS = [_splitmix_sign(n) for n in range(D)]


def _signs(dtype=torch.float32):
    return torch.tensor(SIGNS, dtype=dtype, device="cuda")


def _stage(x, h):
    y = x.view(x.shape[0], D // (2 * h), 2, h)
    return torch.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], dim=2).view(x.shape)


def hadamard(x):
    for h in (1, 2, 4, 8, 16, 32, 64):
        x = _stage(x, h)
    return x


def _half_bytes(d):
    return d.to(torch.float16).view(torch.uint8).view(*d.shape, 2)


def _levels(x):
    """The 4-bit rule over the last dimension: levels 0..15 and the scale."""
    size = x.abs()
    at = torch.where(size == size.amax(-1, keepdim=True), torch.arange(x.shape[-1], device="cuda"), x.shape[-1])
    d = x.gather(-1, at.amin(-1, keepdim=True)) / -8.0
    t = torch.where(d == 0, torch.zeros_like(x), x / d)
    return torch.clamp(torch.trunc(t + 8.5), max=15.0).to(torch.uint8), d


def pack(x, codec):
    """fp32 rows [n][128] as canonical bytes [n][row bytes]."""
    n = x.shape[0]
    if codec == F16:
        return x.to(torch.float16).view(torch.uint8).view(n, 256)
    if codec == Q8_0:
        x = x.reshape(n, 4, 32)
        d = x.abs().amax(-1, keepdim=True) / torch.full((1,), 127.0, device="cuda")
        t = torch.where(d == 0, torch.zeros_like(x), x / d)
        size = t.abs()
        low = torch.floor(size)
        q = torch.copysign(low + ((size - low) >= 0.5).to(torch.float32), t)
        return torch.cat([_half_bytes(d).view(n, 4, 2), q.to(torch.int8).view(torch.uint8)], dim=-1).view(n, 136)
    if codec == Q4_0:
        q, d = _levels(x.reshape(n, 4, 32))
        return torch.cat([_half_bytes(d).view(n, 4, 2), q[..., :16] | (q[..., 16:] << 4)], dim=-1).view(n, 72)
    q, d = _levels(hadamard(x * _signs()) * 0.125)
    q = q.view(n, 4, 32)
    return torch.cat([_half_bytes(d).view(n, 2), (q[..., :16] | (q[..., 16:] << 4)).view(n, 64)], dim=-1)


def unpack(b, codec):
    """Canonical bytes [n][row bytes] as the fp32 rows [n][128] that they stand for."""
    n = b.shape[0]
    if codec == F16:
        return b.contiguous().view(torch.float16).to(torch.float32)
    if codec == Q8_0:
        b = b.reshape(n, 4, 34)
        d = b[..., :2].contiguous().view(torch.float16).to(torch.float32)
        return (d * b[..., 2:].contiguous().view(torch.int8).to(torch.float32)).view(n, D)
    if codec == Q4_0:
        b = b.reshape(n, 4, 18)
        d = b[..., :2].contiguous().view(torch.float16).to(torch.float32)
        q = torch.cat([b[..., 2:] & 15, b[..., 2:] >> 4], dim=-1).to(torch.float32) - 8.0
        return (d * q).view(n, D)
    d = b[:, :2].contiguous().view(torch.float16).to(torch.float32)
    b = b[:, 2:].reshape(n, 4, 16)
    q = torch.cat([b & 15, b >> 4], dim=-1).to(torch.float32).view(n, D) - 8.0
    return hadamard(d * q) * 0.0625 * _signs()


# ------------------------------------------------------------------------------------- inputs

def _random(shape, seed, k, dtype=torch.float16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + k)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(sizes):
    return _ints([sum(sizes[:i]) for i in range(len(sizes) + 1)])


def _caches(case, lens, codecs, seed, fill=True):
    """One layer's two sides with tokens of N(0, 1), contiguous or in shuffled pages."""
    c = dict(n_seqs=len(lens), n_kv=case["n_kv"], codecs=codecs, lens=_ints(lens), table=None, n_pages=0)
    c["capacity"] = max(256, -(-max(lens) // 256) * 256)
    if case["paged"]:
        per = c["capacity"] // 256
        c["n_pages"] = c["n_seqs"] * per + 3
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 1009 + 77)
        table = torch.randperm(c["n_pages"], generator=g, device="cuda")[: c["n_seqs"] * per]
        c["table"] = table.to(torch.int32).view(c["n_seqs"], per)
    tokens = c["n_pages"] * 256 if case["paged"] else c["n_seqs"] * c["capacity"]
    n, c["sides"] = tokens * case["n_kv"] // 16, []
    for side, codec in enumerate(codecs):
        if not fill:
            c["sides"].append(torch.zeros(n * 16 * ROW[codec], dtype=torch.uint8, device="cuda"))
        elif codec == F16:
            c["sides"].append(_random((n * 16 * D,), seed, 20 + side).view(torch.uint8))
        else:
            rows = pack(_random((n * 16, D), seed, 20 + side).to(torch.float32), codec)
            cache = torch.empty((n, 16 * ROW[codec]), dtype=torch.uint8, device="cuda")
            cache[:, offsets(codec, side).reshape(-1)] = rows.view(n, -1)
            c["sides"].append(cache.view(-1))
    return c


def _layer(c, n_q):
    """What a user's program keeps beside its buffers: the layer's descriptor over them."""
    import attention_quantized_kv_gb300 as kvq
    made = kvq.KVLayer(c["n_seqs"], c["n_kv"], n_q, c["capacity"], *c["codecs"], k_cache=c["sides"][0],
                       v_cache=c["sides"][1], n_pages=c["n_pages"], block_table=c["table"])
    made.seq_lens = c["lens"]
    return made


def _workspace(nbytes):
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    op, s, codecs = case["op"], {"case": case}, (case["k"], case["v"])
    if own:
        import attention_quantized_kv_gb300 as kvq
        s["kvq"] = kvq
    if op in ("prefix", "cross"):
        rows, n_q, kind = case["seqs"] if op == "prefix" else case["rows"], case["n_q"], TYPES[case.get("type", "f16")]
        s["q"] = _random((rows, n_q, D), seed, 1, kind)
        s["out"] = torch.empty_like(s["q"])
        s["cache"] = _caches(case, lengths(case), codecs, seed)
        if op == "prefix":
            s["prefix"] = _caches(case, prefixes(case), (case["pk"], case["pv"]), seed + 500009)
            s["group_start"] = _starts(shares(case["seqs"], case["groups"]))
        else:
            s["row_start"] = _starts(counts(case))
        if own:
            s["layer"] = _layer(s["cache"], n_q)
            longest = max(lengths(case))
            if op == "prefix":
                s["shared"] = _layer(s["prefix"], n_q)
                s["work"] = _workspace(kvq.attn_decode_prefix_workspace(s["layer"], s["shared"], longest, case["prefix"]))
            else:
                s["work"] = _workspace(kvq.attn_cross_workspace(s["layer"], rows, longest))
        return s
    new, lens = counts(case), lengths(case)
    total, n_kv = sum(new), case["n_kv"]
    s["row_start"] = _starts(new)
    s["k"], s["v"] = (torch.empty((total, n_kv, D), dtype=TYPES[case["type"]], device="cuda") for _ in "kv")
    if op == "append":
        s["cache"] = _caches(case, [a + b for a, b in zip(lens, new)], codecs, seed, fill=False)
        s["kv"] = _random((total, 2 * n_kv, D), seed, 1, TYPES[case["type"]])
        s["cache"]["lens"], s["before"], s["after"] = _ints(lens), _ints(lens), _ints([a + b for a, b in zip(lens, new)])
    else:
        s["cache"] = _caches(case, lens, codecs, seed)
        s["before"] = _ints([a - b for a, b in zip(lens, new)])  # the last tokens of each
    if own:
        s["layer"] = _layer(s["cache"], n_kv)
        if op == "append":
            s["reader"] = _layer(dict(s["cache"], lens=s["after"]), n_kv)
    return s


# ------------------------------------------------------------------------------------- the plain forms

def side_values(c, side, seq, length):
    """fp32 [kv heads][length][128] of one sequence of a cache side."""
    codec, t = c["codecs"][side], torch.arange(length, device="cuda")
    u = units(torch.full_like(t, seq)[None], torch.arange(c["n_kv"], device="cuda")[:, None], t[None], c["n_kv"],
              c["capacity"], c["table"])
    b = row_bytes_at(c["sides"][side], codec, side, u, (t % 16)[None].expand(u.shape))
    return unpack(b.view(-1, ROW[codec]), codec).view(c["n_kv"], length, D)


def softmax_parts(q, c, seq, length):
    """Rows q [kv heads][n][128] against one sequence: the running maximum, sum and weighted sum."""
    a = torch.matmul(q, side_values(c, 0, seq, length).transpose(-1, -2)) * SCALE
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - top)
    return top, p.sum(-1, keepdim=True), torch.matmul(p, side_values(c, 1, seq, length))


def as_heads(q, n_kv):
    """[n][n_q][128] as [kv heads][n * group][128] in fp32."""
    n, n_q = q.shape[:2]
    return q.to(torch.float32).view(n, n_kv, n_q // n_kv, D).transpose(0, 1).reshape(n_kv, -1, D)


def as_rows(x, n):
    """[kv heads][n * group][w] as [n][n_q][w]."""
    return x.view(x.shape[0], n, -1, x.shape[-1]).transpose(0, 1).reshape(n, -1, x.shape[-1])


def plain_cross(s):
    c, case, at = s["cache"], s["case"], 0
    for i, (n, length) in enumerate(zip(counts(case), lengths(case))):
        top, total, o = softmax_parts(as_heads(s["q"][at:at + n], c["n_kv"]), c, i, length)
        s["out"][at:at + n] = as_rows(o / total, n).to(s["out"].dtype)
        at += n
    return s["out"]


def plain_prefix(s):
    c, case, at = s["cache"], s["case"], 0
    own_lengths = lengths(case)
    for g, (n, length) in enumerate(zip(shares(case["seqs"], case["groups"]), prefixes(case))):
        shared = [as_rows(x, n) for x in softmax_parts(as_heads(s["q"][at:at + n], c["n_kv"]), s["prefix"], g, length)]
        for i in range(n):
            mine = softmax_parts(as_heads(s["q"][at + i:at + i + 1], c["n_kv"]), c, at + i, own_lengths[at + i])
            top, total, o = (as_rows(x, 1)[0] for x in mine)
            m = torch.maximum(top, shared[0][i])
            a, b = torch.exp(top - m), torch.exp(shared[0][i] - m)
            total = total * a + shared[1][i] * b
            s["out"][at + i] = ((o * a + shared[2][i] * b) / total).to(torch.float16)
        at += n
    return s["out"]


def _places(s, first):
    """(unit, row) [rows][kv heads] of the packed rows whose sequences begin at token `first`."""
    c, start = s["cache"], s["row_start"].long()
    at = torch.arange(sum(counts(s["case"])), device="cuda")
    seq = torch.searchsorted(start, at, right=True) - 1
    pos = first.long()[seq] + at - start[seq]
    u = units(seq[:, None], torch.arange(c["n_kv"], device="cuda")[None], pos[:, None], c["n_kv"], c["capacity"], c["table"])
    return u, (pos % 16)[:, None].expand(u.shape)


def plain_rows(s):
    case, c = s["case"], s["cache"]
    got = {}
    if case["op"] == "append" and case["update"]:
        c["lens"].copy_(s["before"])
    unit, row = _places(s, c["lens"] if case["op"] == "append" else s["before"])
    for side, name in enumerate("kv"):
        codec, cache = c["codecs"][side], c["sides"][side]
        if case["op"] == "append":
            x = s["kv"][:, side * c["n_kv"]:(side + 1) * c["n_kv"]].to(torch.float32)
            data = pack(x.reshape(-1, D), codec).view(*unit.shape, -1)
            cache[unit[..., None] * (16 * ROW[codec]) + offsets(codec, side)[row]] = data
        b = row_bytes_at(cache, codec, side, unit, row)
        s[name].copy_(unpack(b.view(-1, ROW[codec]), codec).view(*unit.shape, D))
        got[name] = s[name]
    if case["op"] == "append":
        if case["update"]:
            c["lens"].add_(s["row_start"][1:] - s["row_start"][:-1])
        got["lens"] = c["lens"]
    return got


# ------------------------------------------------------------------------------------- a pass

def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"cross": plain_cross, "prefix": plain_prefix}.get(op, plain_rows)(s)
    kvq, layer = s["kvq"], s["layer"]
    if op == "cross":
        # one row for each sequence is the call's default
        start = None if case["rows"] == case["seqs"] else s["row_start"]
        kvq.attn_cross(layer, s["q"], SCALE, s["out"], None, max(lengths(case)), s["work"], row_start=start)
        return s["out"]
    if op == "prefix":
        kvq.attn_decode_prefix(layer, s["shared"], s["q"], SCALE, s["out"], None, max(lengths(case)), case["prefix"],
                               s["work"], group_start=s["group_start"])
        return s["out"]
    if op == "read":
        kvq.kv_read_rows(layer, s["k"], s["v"], row_start=s["row_start"], first=s["before"])
        return {"k": s["k"], "v": s["v"]}
    if case["update"]:
        s["cache"]["lens"].copy_(s["before"])
    k, v = s["kv"].split(case["n_kv"], dim=1)
    kvq.kv_append_rows(layer, k, v, row_start=s["row_start"], update_lens=case["update"])
    kvq.kv_read_rows(s["reader"], s["k"], s["v"], row_start=s["row_start"], first=s["before"])
    return {"k": s["k"], "v": s["v"], "lens": s["cache"]["lens"]}


# ------------------------------------------------------------------------------------- in 64 bits

def _matrix():
    i = torch.arange(D, device="cuda")
    bits = sum(((i[:, None] & i[None, :]) >> k) & 1 for k in range(7))
    return 1.0 - 2.0 * (bits % 2).double()


def _rows64(c, side, seq, pos):
    """fp64 [kv heads][n][128]: the values of one sequence's tokens `pos`, from the codes."""
    codec, n_kv = c["codecs"][side], c["n_kv"]
    head = torch.arange(n_kv, device="cuda")[:, None]
    page = None if c["table"] is None else c["table"][seq].long()[pos // 256]
    unit = (seq * n_kv + head) * (c["capacity"] // 16) + pos // 16 if page is None else \
        (page * n_kv + head) * 16 + pos % 256 // 16
    place = torch.from_numpy(np.ascontiguousarray(unit_offsets(codec, side))).cuda()[pos % 16]
    b = c["sides"][side][unit[..., None] * (16 * ROW[codec]) + place]
    if codec == F16:
        return b.view(torch.float16).double()
    blocks = 1 if codec == TURBO4 else 4
    b = b.view(n_kv, len(pos), blocks, ROW[codec] // blocks)
    scale, code = b[..., :2].contiguous().view(torch.float16).double(), b[..., 2:]
    if codec == Q8_0:
        return (code.contiguous().view(torch.int8).double() * scale).flatten(-2)
    code = code.reshape(n_kv, len(pos), 4, 16)
    y = (torch.cat([code % 16, code // 16], dim=-1).double() - 8) * scale
    return y.flatten(-2) if codec == Q4_0 else y.flatten(-2) @ _matrix() / 16 * _signs(torch.float64)


def _held(x, codec):
    """The values that a codec holds for fp64 rows [..., 128], by its rule in 64 bits."""
    if codec == F16:
        return x.to(torch.float16).double()
    y = (x * _signs(torch.float64)) @ _matrix() / 8 if codec == TURBO4 else x
    y = y.unflatten(-1, (-1, D if codec == TURBO4 else 32))
    if codec == Q8_0:
        d = y.abs().amax(-1, keepdim=True) / 127
        q = torch.where(d == 0, torch.zeros_like(y), torch.sign(y) * torch.floor((y / d).abs() + 0.5))
    else:
        big = y.gather(-1, (y.abs() == y.abs().amax(-1, keepdim=True)).double().argmax(-1, keepdim=True))
        d = big / -8
        q = torch.where(d == 0, torch.zeros_like(y), torch.clamp(torch.floor(y / d + 8.5), max=15.0) - 8)
    v = (d.to(torch.float16).double() * q).flatten(-2)
    return v @ _matrix() / 16 * _signs(torch.float64) if codec == TURBO4 else v


def exact(case, seed):
    s = prepare(case, seed)
    c, op, lens = s["cache"], case["op"], lengths(case)
    if op in ("append", "read"):
        got = {}
        for side, name in enumerate("kv"):
            if op == "append":
                x = s["kv"][:, side * c["n_kv"]:(side + 1) * c["n_kv"]].double()
                got[name] = _held(x, c["codecs"][side])
            else:
                got[name] = torch.cat([_rows64(c, side, i, torch.arange(n - m, n, device="cuda")).transpose(0, 1)
                                       for i, (n, m) in enumerate(zip(lens, counts(case)))])
        return dict(got, lens=None) if op == "append" else got
    group, q = case["n_q"] // case["n_kv"], s["q"].double()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    sizes = counts(case) if op == "cross" else shares(case["seqs"], case["groups"])
    shared = (c, lens) if op == "cross" else (s["prefix"], prefixes(case))
    at = 0
    for g, (n, length) in enumerate(zip(sizes, shared[1])):
        # every row of the group over the keys that all of its rows see, and over its sequence's own
        pieces = [(slice(at, at + n), shared[0], g, length)]
        if op == "prefix":
            pieces += [(slice(i, i + 1), c, i, lens[i]) for i in range(at, at + n)]
        sides = [[_rows64(p, side, i, torch.arange(m, device="cuda")) for _, p, i, m in pieces] for side in (0, 1)]
        for h in range(case["n_kv"]):
            heads = slice(h * group, (h + 1) * group)
            a = [torch.einsum("ngd,td->ngt", q[rows, heads], k[h]) / math.sqrt(D)
                 for (rows, *_), k in zip(pieces, sides[0])]
            total = torch.logsumexp(a[0], -1)
            if op == "prefix":
                total = torch.logaddexp(total, torch.cat([torch.logsumexp(x, -1) for x in a[1:]]))
            lse[at:at + n, heads] = total
            out[at:at + n, heads] = 0
            for (rows, *_), x, v in zip(pieces, a, sides[1]):
                out[rows, heads] += torch.einsum("ngt,td->ngd", torch.exp(x - lse[rows, heads][..., None]), v[h])
        at += n
    return out
