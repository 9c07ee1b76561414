"""The rotary-position operators, as they are measured: each in a plain form of elementary torch
operations, and as the calls that a user makes of the library.

  table   the (cos, sin) table of every position, with its frequencies scaled for long contexts
  apply   the rotation of query rows, or its transpose (the gradient)
  append  new keys (rotated) and values encoded into the cache, the queries rotated beside them
  shift   cached keys rotated again after an eviction moved them to other positions
  decode  one decode step: query and new key rotated, token appended, all keys attended

Every operator but `table` takes the same fp32 table on both sides.  A rotation is
(RN(RN(a c) - RN(b s)), RN(RN(a s) + RN(b c))) in fp32, so caches and rotated rows are the same bit
for bit.  A cache side held in fewer than 16 bits is returned as fp16 values (read back through the
library's re-encode call), in the order of the f16 cache.
"""
import math

import numpy as np
import torch

own = False

D = 128
F16, Q8_0, Q4_0, TURBO4 = 0, 1, 2, 3
ROW = {F16: 256, Q8_0: 136, Q4_0: 72, TURBO4: 66}
BITS = {F16: 16, Q8_0: 8, Q4_0: 4, TURBO4: 4}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SCALINGS = ("plain", "linear", "ntk", "parts", "yarn")


# ------------------------------------------------------------------------------------- cases

def listed():
    rope = {"layout": "half", "rot": 128, "magnitude": 1.0}
    return [
        # a server builds the table of its slots' length once, when it loads a model
        dict(name="angles for 32768 positions", op="table", n_pos=32768, rot=128, scaling="plain",
             base=10000.0, factor=1.0, orig=32768),
        # the longest slot of the repository's workloads, its context stretched four times
        dict(name="angles for 200704 positions", op="table", n_pos=200704, rot=128, scaling="yarn",
             base=1000000.0, factor=4.0, orig=50176),
        # the query of the eviction probe: one row per sequence, launch latency
        dict(name="probe queries of 16 slots", op="apply", rows=16, heads=40, type="f16",
             n_pos=65536, transpose=False, extra=0, **rope),
        # the gradient of a long prompt's queries, a view of a fused projection, part of the head
        dict(name="gradient of 8191 query rows", op="apply", rows=8191, heads=40, type="bf16",
             n_pos=8192, transpose=True, extra=16, **dict(rope, layout="interleaved", rot=64)),
        # one token for each of 16 slots: the append of every layer of a decode step
        dict(name="append 16 single tokens", op="append", seqs=16, prompts=0, tokens=16, past=2047,
             n_q=40, n_kv=8, k=F16, v=F16, type="f16", paged=True, update=False, **rope),
        # the first ubatch of a prompt into 8-bit caches
        dict(name="append a 2048-token ubatch", op="append", seqs=1, prompts=1, tokens=2048, past=0,
             n_q=32, n_kv=8, k=Q8_0, v=Q8_0, type="f16", paged=False, update=False, **rope),
        # prompts of odd lengths among single tokens, bf16 projections, part of the head, scaled
        dict(name="append a mixed batch", op="append", seqs=24, prompts=4, tokens=1821, past=701,
             n_q=40, n_kv=8, k=F16, v=F16, type="bf16", paged=True, update=True, layout="interleaved",
             rot=96, magnitude=1.1386294361119891),
        # four long prompts at once under the asymmetric contract (K f16, V q8_0)
        dict(name="append 32768 prompt tokens", op="append", seqs=4, prompts=4, tokens=32768, past=0,
             n_q=32, n_kv=4, k=F16, v=Q8_0, type="f16", paged=False, update=False, **rope),
        # keys of four long slots after an eviction took cells out of their middle
        dict(name="shift f16 keys of long slots", op="shift", seqs=4, n_kv=8, past=32768, gone=2048,
             k=F16, paged=False, **rope),
        # the same for short paged slots with 8-bit keys
        dict(name="shift q8_0 keys of short slots", op="shift", seqs=8, n_kv=8, past=4097, gone=511,
             k=Q8_0, paged=True, **rope),
        # a decode step of a short slot: latency
        dict(name="decode step at 4096 keys", op="decode", seqs=1, n_q=8, n_kv=2, past=4096, k=Q8_0,
             v=Q8_0, paged=True, **rope),
        # a decode step of two long slots, one of them filled by it
        dict(name="decode step at 200703 keys", op="decode", seqs=2, n_q=32, n_kv=4, past=200703, k=F16,
             v=F16, paged=False, **rope),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["table", "apply", "append", "append", "shift", "decode"])
    rope = {"layout": rng.choice(["half", "interleaved"]),
            "rot": rng.choice([128, 128, 96, 64, 32, 2 * rng.randint(1, 64)]),
            "magnitude": rng.choice([1.0, 1.0, 1.0 + 0.1 * math.log(rng.uniform(1.5, 32.0))])}
    if op == "table":
        factor = rng.uniform(1.0, 16.0)
        n_pos = _log(rng, 1, 200704)
        return dict(op=op, n_pos=n_pos, rot=max(4, rope["rot"]), scaling=rng.choice(SCALINGS),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), factor=factor,
                    orig=max(64, int(n_pos / factor)))
    if op == "apply":
        return dict(op=op, rows=_log(rng, 1, 16384), heads=rng.choice([1, 2, 5, 8, 12, 32, 40]),
                    type=rng.choice(["f16", "bf16", "f32"]), n_pos=rng.randint(1, 65536),
                    transpose=rng.random() < 0.5, extra=rng.choice([0, 0, 1, 16]), **rope)
    n_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 5, 8])
    k, v = rng.choice([F16, F16, Q8_0, Q4_0, TURBO4]), rng.choice([F16, F16, Q8_0, Q4_0, TURBO4])
    if op == "append":
        seqs = _log(rng, 1, 64)
        prompts = rng.randint(0, min(seqs, 4))
        tokens = seqs - prompts + (_log(rng, prompts, 16384) if prompts else 0)
        return dict(op=op, seqs=seqs, prompts=prompts, tokens=tokens,
                    past=rng.choice([0, rng.randint(1, 2048)]), n_q=n_kv * group, n_kv=n_kv, k=k, v=v,
                    type=rng.choice(["f16", "bf16", "f32"]), paged=rng.random() < 0.5,
                    update=rng.random() < 0.5, **rope)
    if op == "shift":
        past = _log(rng, 2, 32768)
        return dict(op=op, seqs=rng.choice([1, 2, 3, 4]), n_kv=n_kv, past=past,
                    gone=rng.randint(1, max(1, past // 4)), k=k, paged=rng.random() < 0.5, **rope)
    return dict(op=op, seqs=rng.choice([1, 2, 3, 7]), n_q=n_kv * group, n_kv=n_kv,
                past=_log(rng, 63, 65536), k=k, v=v, paged=k != F16 or v != F16 or rng.random() < 0.5,
                **rope)


def lengths(case):
    """Cached tokens per sequence before the call: the longest first, the rest spread below it."""
    n = case["seqs"]
    return [case["past"] * (n - s) // n for s in range(n)]


def counts(case):
    """New tokens per sequence of an append: uneven prompts, then one token each."""
    p, n = case["prompts"], case["seqs"]
    rest = case["tokens"] - (n - p)
    shares = [i + 3 for i in range(p)]
    got = [max(1, rest * w // sum(shares)) for w in shares]
    if p:
        got[-1] += rest - sum(got)
    return got + [1] * (n - p)


def evicted(case):
    return [min(case["gone"], max(0, n - 4)) for n in lengths(case)]


def work(case):
    op = case["op"]
    if op == "table":
        pairs = case["n_pos"] * (case["rot"] // 2)
        return {"bytes": pairs * 8, "flops": pairs * 24}
    angles = 4 * case["rot"]
    if op == "apply":
        size = torch.empty(0, dtype=TYPES[case["type"]]).element_size()
        n = case["rows"] * case["heads"]
        return {"bytes": 2 * n * D * size + case["rows"] * (4 + min(angles * case["n_pos"] / case["rows"], angles)),
                "flops": 3 * n * case["rot"]}
    if op == "append":
        size = torch.empty(0, dtype=TYPES[case["type"]]).element_size()
        n, q, kv = case["tokens"], case["n_q"], case["n_kv"]
        back = sum((ROW[c] + 256) * kv * (sum(lengths(case)) + n) for c in (case["k"], case["v"]) if c != F16)
        return {"bytes": n * ((q + 2 * kv) * D * size + q * 256 + kv * (ROW[case["k"]] + ROW[case["v"]]) + angles) + back,
                "flops": 3 * n * (q + kv) * case["rot"]}
    if op == "shift":
        left = [a - b for a, b in zip(lengths(case), evicted(case))]
        rows = sum(left) * case["n_kv"]
        back = rows * (ROW[case["k"]] + 256) if case["k"] != F16 else 0
        return {"bytes": 2 * rows * ROW[case["k"]] + sum(left) * 4 + sum(evicted(case)) * 4 + back, "flops": 3 * rows * case["rot"]}
    keys = sum(n + 1 for n in lengths(case))
    return {"bytes": keys * case["n_kv"] * (ROW[case["k"]] + ROW[case["v"]]) + case["seqs"] * case["n_q"] * 516,
            "flops": 4 * keys * case["n_q"] * D}


# ------------------------------------------------------------------------------------- angles

def frequencies(c):
    """Radians per position of every pair, as Python floats."""
    n, base, factor = c["rot"] // 2, c["base"], c["factor"]
    if c["scaling"] == "ntk" and n > 1:
        base = base * factor ** (c["rot"] / (c["rot"] - 2))
    f = np.power(base, -np.arange(n) * 2.0 / c["rot"])
    if c["scaling"] == "linear":
        f = f / factor
    if c["scaling"] == "parts":  # by the turns that a pair makes over the original length
        turns = c["orig"] * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    if c["scaling"] == "yarn":  # by the index at which a pair makes 32 turns, and one turn
        at = [c["rot"] * math.log(c["orig"] / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
        keep = 1 - np.clip((np.arange(n) - low) / max(high - low, 0.001), 0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    return [float(x) for x in f]


def angle_table(freqs, n_pos, dtype=torch.float32):
    """[n_pos][pairs][2] of cos and sin, the angles of far positions in 64 bits."""
    at = torch.arange(n_pos, dtype=torch.float64, device="cuda")
    f = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    a = at[:, None] * f[None, :]
    return torch.stack([torch.cos(a), torch.sin(a)], dim=-1).to(dtype)


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


def offsets(codec, side):
    return torch.from_numpy(np.ascontiguousarray(unit_offsets(codec, side))).cuda()


def units(seq, head, pos, n_kv, capacity, table):
    """The unit that holds token `pos` of (seq, kv head), in the cache or the page pool."""
    if table is None:
        return (seq * n_kv + head) * (capacity // 16) + pos // 16
    return (table[seq, pos // 256].long() * n_kv + head) * 16 + (pos // 16) % 16


def put_rows(cache, codec, side, unit, row, data):
    """Rows of canonical bytes into their places: unit, row [...], data [..., row bytes]."""
    cache[unit[..., None] * (16 * ROW[codec]) + offsets(codec, side)[row]] = data


def all_rows(cache, codec, side):
    """[units][16][row bytes]: every row of a cache, in canonical order."""
    u = cache.view(-1, 16 * ROW[codec])
    return u[:, offsets(codec, side).reshape(-1)].view(-1, 16, ROW[codec])


def as_f16_cache(values, side):
    """Values [units][16][128] as the f16 cache that would hold them, as a flat fp16 tensor."""
    to = torch.empty(16 * 256, dtype=torch.int64, device="cuda")
    to[offsets(F16, side).reshape(-1)] = torch.arange(16 * 256, device="cuda")
    return values.to(torch.float16).view(torch.uint8).view(-1, 16 * 256)[:, to].contiguous().view(-1).view(torch.float16)


# ------------------------------------------------------------------------------------- codecs

def _splitmix_sign(n):
    z = (0x4B5651 + 0x9E3779B97F4A7C15 * (n + 1)) & (2**64 - 1)
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & (2**64 - 1)
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & (2**64 - 1)
    return -1.0 if ((z ^ (z >> 31)) >> 63) & 1 else 1.0


SIGNS = [_splitmix_sign(n) for n in range(D)]


def _stage(x, h):
    y = x.view(x.shape[0], D // (2 * h), 2, h)
    return torch.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], dim=2).view(x.shape)


def hadamard(x):
    x = _stage(_stage(_stage(x, 1), 2), 4)
    return _stage(_stage(_stage(_stage(x, 8), 16), 32), 64)


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
    q, d = _levels(hadamard(x * torch.tensor(SIGNS, device="cuda")) * 0.125)
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
    return hadamard(d * q) * 0.0625 * torch.tensor(SIGNS, device="cuda")


# ------------------------------------------------------------------------------------- inputs

def _random(shape, seed, k, dtype=torch.float16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + k)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(case, capacity, seed):
    """Block table and pool size: every page of every sequence on a pool page of its own, shuffled."""
    if not case["paged"]:
        return None, 0
    per = capacity // 256
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1009 + 77)
    n = case["seqs"] * per + 3
    return torch.randperm(n, generator=g, device="cuda")[: case["seqs"] * per].to(torch.int32).view(case["seqs"], per), n


def _cache(case, codec, side, capacity, n_pages, seed):
    """A filled cache (or pool): rows of N(0, 1)."""
    n = (n_pages * 256 if n_pages else case["seqs"] * capacity) * case["n_kv"] // 16
    if codec == F16:
        return _random((n * 16 * D,), seed, 20 + side).view(torch.uint8)
    rows = pack(_random((n * 16, D), seed, 20 + side).to(torch.float32), codec).view(n, 16, ROW[codec])
    cache = torch.empty(n * 16 * ROW[codec], dtype=torch.uint8, device="cuda")
    cache.view(n, -1)[:, offsets(codec, side).reshape(-1)] = rows.view(n, -1)
    return cache


def _zeros(case, codec, capacity, n_pages):
    n = (n_pages * 256 if n_pages else case["seqs"] * capacity) * case["n_kv"]
    return torch.zeros(n * ROW[codec], dtype=torch.uint8, device="cuda")


def _handles(s):
    """What a user's program keeps beside its buffers: the layer and rope descriptors over them."""
    import attention_quantized_kv_gb300 as kvq
    c = s["case"]
    s["kvq"] = kvq
    layout = kvq.KVQ_ROPE_HALF if c["layout"] == "half" else kvq.KVQ_ROPE_INTERLEAVED
    s["rope"] = kvq.Rope(table=s["table"], layout=layout, magnitude=c["magnitude"])
    if c["op"] == "apply":
        return

    def layer(lens, block_table=s["blocks"], capacity=s["capacity"]):
        v, v_codec = (s["v"], c["v"]) if "v" in s else (s["k"], c["k"])
        made = kvq.KVLayer(c["seqs"], c["n_kv"], c.get("n_q", c["n_kv"]), capacity, c["k"], v_codec,
                           k_cache=s["k"], v_cache=v, n_pages=s["n_pages"], block_table=block_table)
        made.seq_lens = lens
        return made

    s["layer"] = layer(s["lens"])
    s["after"] = layer(s["lens_after"])
    if c["op"] == "decode":
        s["work"] = torch.zeros(kvq.attn_decode_workspace(s["layer"], s["capacity"]), dtype=torch.uint8, device="cuda")
        if c["paged"]:  # the one page of each sequence that the step writes to
            s["after"] = layer(s["last_lens"], s["last_page"], 256)


def prepare(case, seed):
    op, s = case["op"], {"case": case}
    if op == "table":
        # the only input is a list of plain numbers: the seed moves the base of the frequencies
        s["case"] = dict(case, base=case["base"] * (1 + (seed % 1000003) * 1e-9))
        s["out"] = torch.empty((case["n_pos"], case["rot"] // 2, 2), dtype=torch.float32, device="cuda")
        return s
    rope = dict(case, scaling="plain", base=500000.0, factor=1.0)
    if op == "apply":
        wide = _random((case["rows"], case["heads"] + case["extra"], D), seed, 1, TYPES[case["type"]])
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 1009 + 5)
        s["x"] = wide[:, : case["heads"]]
        s["positions"] = torch.randint(0, case["n_pos"], (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
        s["y"] = torch.empty((case["rows"], case["heads"], D), dtype=TYPES[case["type"]], device="cuda")
        s["table"] = angle_table(frequencies(rope), case["n_pos"])
        if own:
            _handles(s)
        return s
    lens = lengths(case)
    new = counts(case) if op == "append" else [1] * case["seqs"] if op == "decode" else [0] * case["seqs"]
    s["capacity"] = max(256, -(-max(a + b for a, b in zip(lens, new)) // 256) * 256)
    s["blocks"], s["n_pages"] = _pages(case, s["capacity"], seed)
    s["lens"], s["lens_before"] = _ints(lens), _ints(lens)
    s["table"] = angle_table(frequencies(rope), s["capacity"])
    if op == "append":
        heads = case["n_q"] + 2 * case["n_kv"]
        s["qkv"] = _random((case["tokens"], heads, D), seed, 1, TYPES[case["type"]])
        s["row_start"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
        s["q_out"] = torch.empty((case["tokens"], case["n_q"], D), dtype=torch.float16, device="cuda")
        s["k"], s["v"] = (_zeros(case, case[c], s["capacity"], s["n_pages"]) for c in "kv")
        s["lens_after"] = _ints([a + b for a, b in zip(lens, new)])
    elif op == "shift":
        gone = evicted(case)
        g = np.random.RandomState(seed % (2**32))
        rows = np.zeros((case["seqs"], max(1, max(gone))), np.int32)
        for i, (n, e) in enumerate(zip(lens, gone)):
            rows[i, :e] = np.sort(g.permutation(np.arange(4, n))[:e])
        s["evict"], s["n_evicted"] = torch.from_numpy(rows).cuda(), _ints(gone)
        s["delta"] = torch.zeros((case["seqs"], s["capacity"]), dtype=torch.int32, device="cuda")
        s["k"] = _cache(case, case["k"], 0, s["capacity"], s["n_pages"], seed)
        s["lens_after"] = _ints([a - b for a, b in zip(lens, gone)])
    else:
        s["q"] = _random((case["seqs"], case["n_q"], D), seed, 1)
        s["k_new"], s["v_new"] = (_random((case["seqs"], case["n_kv"], D), seed, 2 + i) for i in (0, 1))
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["seqs"], case["n_q"]), dtype=torch.float32, device="cuda")
        s["k"], s["v"] = (_cache(case, case[c], i, s["capacity"], s["n_pages"], seed) for i, c in enumerate("kv"))
        s["lens_after"] = _ints([a + 1 for a in lens])
        if case["paged"]:
            s["last_page"] = torch.stack([s["blocks"][i, n // 256] for i, n in enumerate(lens)]).view(-1, 1).contiguous()
            s["last_lens"] = _ints([n % 256 + 1 for n in lens])
    for i, c in enumerate("kv"):
        if c in s and case[c] != F16:
            s["back_" + c] = torch.zeros(s[c].numel() // ROW[case[c]] * 256, dtype=torch.uint8, device="cuda")
    if own:
        _handles(s)
    return s


# ------------------------------------------------------------------------------------- the plain forms

def rotate(x, cs, c, sign=1.0):
    """Rows x [n][heads][128] in fp32 by the table rows cs [n][rot / 2][2] (or [n][heads][rot / 2][2])."""
    n = c["rot"] // 2
    cs = cs if cs.dim() == 4 else cs[:, None]
    co, si = cs[..., 0], cs[..., 1] * sign
    if c["layout"] == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        return torch.cat([a * co - b * si, a * si + b * co, x[..., 2 * n:]], dim=-1)
    a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    return torch.cat([torch.stack([a * co - b * si, a * si + b * co], dim=-1).flatten(-2), x[..., 2 * n:]], dim=-1)


def angles_at(s, positions):
    return s["table"][positions.long()] * s["case"]["magnitude"]


def read_back(s, side, lens, block_table, capacity):
    """The fp16 values that a cache side stands for, below the lengths, in the order of an f16 cache."""
    c, name = s["case"], "kv"[side]
    if c[name] == F16:
        return s[name].view(torch.float16)
    values = unpack(all_rows(s[name], c[name], side).view(-1, ROW[c[name]]), c[name]).view(-1, 16, D)
    t = torch.arange(capacity, device="cuda")
    seq, head = torch.arange(c["seqs"], device="cuda")[:, None, None], torch.arange(c["n_kv"], device="cuda")[None, :, None]
    u = units(seq, head, t[None, None, :], c["n_kv"], capacity, block_table)
    live = torch.zeros((values.shape[0], 16), dtype=torch.bool, device="cuda")
    live[u, t % 16] = (t[None, None, :] < lens[:, None, None]).expand(u.shape)
    return as_f16_cache(torch.where(live[..., None], values, torch.zeros_like(values)), side)


def plain_append(s):
    c = s["case"]
    n_q, n_kv, total = c["n_q"], c["n_kv"], c["tokens"]
    if c["update"]:
        s["lens"].copy_(s["lens_before"])
    at = torch.arange(total, device="cuda")
    seq = torch.searchsorted(s["row_start"].long(), at, right=True) - 1
    pos = s["lens"].long()[seq] + at - s["row_start"].long()[seq]
    x, cs = s["qkv"].to(torch.float32), angles_at(s, pos)
    q = rotate(x[:, :n_q], cs, c).to(torch.float16)
    k, v = rotate(x[:, n_q:n_q + n_kv], cs, c), x[:, n_q + n_kv:]
    head = torch.arange(n_kv, device="cuda")[None, :].expand(total, n_kv)
    u = units(seq[:, None], head, pos[:, None], n_kv, s["capacity"], s["blocks"])
    row = (pos % 16)[:, None].expand(total, n_kv)
    put_rows(s["k"], c["k"], 0, u, row, pack(k.reshape(-1, D), c["k"]).view(total, n_kv, -1))
    put_rows(s["v"], c["v"], 1, u, row, pack(v.reshape(-1, D), c["v"]).view(total, n_kv, -1))
    if c["update"]:
        s["lens"].add_((s["row_start"][1:] - s["row_start"][:-1]))
    back = [read_back(s, i, s["lens_after"], s["blocks"], s["capacity"]) for i in (0, 1)]
    return {"q": q, "k": back[0], "v": back[1], "lens": s["lens"]}


def plain_shift(s):
    c, cap = s["case"], s["capacity"]
    w = torch.arange(cap, device="cuda").expand(c["seqs"], cap).contiguous()
    j = torch.arange(s["evict"].shape[1], device="cuda")[None, :]
    # cell w came from w + (the evicted cells at or below it): evict[j] - j is non-decreasing
    key = torch.where(j < s["n_evicted"][:, None], s["evict"].long() - j, torch.full_like(j, 1 << 40))
    moved = torch.searchsorted(key.contiguous(), w, right=True)
    live = w < s["lens_after"][:, None]
    s["delta"].copy_(torch.where(live, -moved, s["delta"].long()))
    seq, head = torch.arange(c["seqs"], device="cuda")[:, None, None], torch.arange(c["n_kv"], device="cuda")[None, :, None]
    u = units(seq, head, w[:, None, :], c["n_kv"], cap, s["blocks"])
    rows = s["k"][u[..., None] * (16 * ROW[c["k"]]) + offsets(c["k"], 0)[w % 16][:, None]]
    x = unpack(rows.view(-1, ROW[c["k"]]), c["k"]).view(c["seqs"], c["n_kv"], cap, D).transpose(1, 2)
    d = s["delta"].long()
    cs = s["table"][d.abs()]
    cs = torch.stack([cs[..., 0], cs[..., 1] * torch.sign(d).to(torch.float32)[..., None]], dim=-1)
    turned = rotate(x.reshape(-1, c["n_kv"], D), cs.view(-1, *cs.shape[2:]), c)
    packed = pack(turned.reshape(-1, D), c["k"]).view(c["seqs"], cap, c["n_kv"], -1).transpose(1, 2)
    change = (live & (d != 0))[:, None, :, None]
    put_rows(s["k"], c["k"], 0, u, (w % 16)[:, None].expand(u.shape), torch.where(change, packed, rows))
    return {"k": read_back(s, 0, s["lens_after"], s["blocks"], cap), "delta": s["delta"]}


def gather_side(s, side):
    """A cache side as fp32 [seqs][kv heads][capacity][128]."""
    c, name, cap = s["case"], "kv"[side], s["capacity"]
    values = unpack(all_rows(s[name], c[name], side).view(-1, ROW[c[name]]), c[name]).view(-1, 16, D)
    t = torch.arange(cap, device="cuda")
    seq, head = torch.arange(c["seqs"], device="cuda")[:, None, None], torch.arange(c["n_kv"], device="cuda")[None, :, None]
    return values[units(seq, head, t[None, None, :], c["n_kv"], cap, s["blocks"]), t % 16]


def plain_decode(s):
    c, cap = s["case"], s["capacity"]
    n_kv, n_seqs = c["n_kv"], c["seqs"]
    s["lens"].copy_(s["lens_before"])
    pos = s["lens"].long()
    cs = angles_at(s, pos)
    q = rotate(s["q"].to(torch.float32), cs, c).to(torch.float16).to(torch.float32)
    k = rotate(s["k_new"].to(torch.float32), cs, c)
    head = torch.arange(n_kv, device="cuda")[None, :].expand(n_seqs, n_kv)
    u = units(torch.arange(n_seqs, device="cuda")[:, None], head, pos[:, None], n_kv, cap, s["blocks"])
    row = (pos % 16)[:, None].expand(n_seqs, n_kv)
    put_rows(s["k"], c["k"], 0, u, row, pack(k.reshape(-1, D), c["k"]).view(n_seqs, n_kv, -1))
    put_rows(s["v"], c["v"], 1, u, row, pack(s["v_new"].to(torch.float32).view(-1, D), c["v"]).view(n_seqs, n_kv, -1))
    s["lens"].add_(1)
    scores = torch.matmul(q.view(n_seqs, n_kv, -1, D), gather_side(s, 0).transpose(-1, -2)) * (1 / math.sqrt(D))
    dead = torch.arange(cap, device="cuda")[None, :] >= s["lens"][:, None]
    scores = torch.where(dead[:, None, None, :], torch.full_like(scores, -math.inf), scores)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    values = torch.where(dead[:, None, :, None], torch.zeros((), device="cuda"), gather_side(s, 1))
    out = (torch.matmul(p, values) / total).to(torch.float16).view(n_seqs, -1, D)
    lse = (top + torch.log(total)).view(n_seqs, -1)
    if c["paged"]:
        back = [read_back(s, i, s["last_lens"], s["last_page"], 256) for i in (0, 1)]
    else:
        back = [s["k"].view(torch.float16), s["v"].view(torch.float16)]
    return {"out": out, "lse": lse, "lens": s["lens"], "k": back[0], "v": back[1]}


def plain(s):
    c = s["case"]
    if c["op"] == "table":
        return angle_table(frequencies(c), c["n_pos"])
    if c["op"] == "apply":
        cs = angles_at(s, s["positions"])
        return rotate(s["x"].to(torch.float32), cs, c, -1.0 if c["transpose"] else 1.0).to(s["x"].dtype)
    return {"append": plain_append, "shift": plain_shift, "decode": plain_decode}[c["op"]](s)


# ------------------------------------------------------------------------------------- a pass

def own_read_back(s, side):
    """A cache side as fp16 values: the f16 cache itself, or the re-encode call that reads it back."""
    name, kvq = "kv"[side], s["kvq"]
    if s["case"][name] == F16:
        return s[name].view(torch.float16)
    kvq.kv_requantize(s["after"], side, kvq.KVQ_F16, s["back_" + name])
    return s["back_" + name].view(torch.float16)


def run(s):
    if not own:
        return plain(s)
    c = s["case"]
    if c["op"] == "table":
        import attention_quantized_kv_gb300 as kvq
        freqs = kvq.kvq_rope_freqs(c["rot"], c["base"], SCALINGS.index(c["scaling"]), c["factor"], c["orig"])
        kvq.kvq_rope_table(freqs, s["out"])
        return s["out"]
    kvq, rope = s["kvq"], s["rope"]
    if c["op"] == "apply":
        kvq.kvq_rope_apply(rope, s["x"], s["y"], positions=s["positions"], transpose=c["transpose"])
        return s["y"]
    if c["op"] == "append":
        if c["update"]:
            s["lens"].copy_(s["lens_before"])
        q, k, v = s["qkv"].split([c["n_q"], c["n_kv"], c["n_kv"]], dim=1)
        kvq.kv_append_rope(s["layer"], rope, k, v, row_start=s["row_start"], q=q, q_out=s["q_out"],
                           update_lens=c["update"])
        return {"q": s["q_out"], "k": own_read_back(s, 0), "v": own_read_back(s, 1), "lens": s["lens"]}
    if c["op"] == "shift":
        kvq.kv_evict_delta(s["layer"], s["evict"], s["n_evicted"], s["delta"])
        kvq.kv_rope_shift(s["after"], rope, s["delta"])
        return {"k": own_read_back(s, 0), "delta": s["delta"]}
    s["lens"].copy_(s["lens_before"])
    kvq.attn_decode_append_rope(s["layer"], rope, s["k_new"], s["v_new"], s["q"], 1 / math.sqrt(D), s["out"],
                                s["lse"], s["capacity"], s["work"])
    return {"out": s["out"], "lse": s["lse"], "lens": s["lens"], "k": own_read_back(s, 0), "v": own_read_back(s, 1)}


# ------------------------------------------------------------------------------------- in 64 bits

def _turn(x, freqs, positions, case, m=1.0, conj=False):
    """Rows x [n][heads][128] in fp64, rotated as complex numbers by position * frequency."""
    n = case["rot"] // 2
    a = positions.double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device="cuda")
    w = torch.polar(torch.full_like(a, m), -a if conj else a)[:, None]
    x = x.double()
    head = x[..., : 2 * n]
    pairs = head.unflatten(-1, (2, n)).transpose(-1, -2) if case["layout"] == "half" else head.unflatten(-1, (n, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
    z = z.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else z.flatten(-2)
    return torch.cat([z, x[..., 2 * n:]], dim=-1)


def _held(x, codec):
    """The values that a codec holds for fp64 rows [..., 128], by its rule in 64 bits."""
    if codec == F16:
        return x
    y, block = x.reshape(-1, D), 32
    if codec == TURBO4:
        i = torch.arange(D, device="cuda")
        bits = torch.zeros((D, D), dtype=torch.int64, device="cuda")
        for k in range(7):
            bits += ((i[:, None] & i[None, :]) >> k) & 1
        h, signs = 1.0 - 2.0 * (bits % 2).double(), torch.tensor(SIGNS, dtype=torch.float64, device="cuda")
        y, block = (y * signs) @ h / 8, D
    y = y.unflatten(-1, (-1, block))
    if codec == Q8_0:
        d = y.abs().amax(-1, keepdim=True) / 127
        q = torch.where(d == 0, torch.zeros_like(y), torch.sign(y) * torch.floor((y / d).abs() + 0.5))
    else:
        low, high = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
        tie = (low == -high)
        first = torch.where(y == high, 1, 0).argmax(-1, keepdim=True) < torch.where(y == low, 1, 0).argmax(-1, keepdim=True)
        d = torch.where(torch.where(tie, first, high > -low), high, low) / -8
        q = torch.where(d == 0, torch.zeros_like(y), torch.clamp(torch.floor(y / d + 8.5), max=15.0) - 8)
    v = (d.to(torch.float16).double() * q).flatten(-2)
    return ((v @ h) / 16 * signs if codec == TURBO4 else v).view(x.shape)


def _in_cache(values, unit, row, side, n_units, into=None):
    """fp64 rows at (unit, row), in the order of an f16 cache."""
    to = torch.from_numpy(np.ascontiguousarray(unit_offsets(F16, side)[:, ::2] // 2)).cuda()
    cache = torch.zeros(n_units * 16 * D, dtype=torch.float64, device="cuda") if into is None else into
    cache[unit[..., None] * (16 * D) + to[row]] = values
    return cache


def _read(cache, codec, side, unit, row):
    """The fp64 values of the rows at (unit, row) of a cache."""
    b = cache[unit[..., None] * (16 * ROW[codec]) + offsets(codec, side)[row]]
    return unpack(b.view(-1, ROW[codec]), codec).double().view(*unit.shape, D)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    if op == "table":
        return angle_table(frequencies(c), c["n_pos"], torch.float64)
    freqs = frequencies(dict(case, scaling="plain", base=500000.0, factor=1.0))
    if op == "apply":
        return _turn(s["x"], freqs, s["positions"], c, c["magnitude"], c["transpose"])
    n_kv, cap, n_seqs = c["n_kv"], s["capacity"], c["seqs"]
    n_units = s["k"].numel() // (16 * ROW[c["k"]])
    head = torch.arange(n_kv, device="cuda")
    if op == "append":
        new, lens = counts(c), lengths(c)
        seq = torch.repeat_interleave(torch.arange(n_seqs, device="cuda"), torch.tensor(new, device="cuda"))
        pos = torch.cat([torch.arange(a, a + b, device="cuda") for a, b in zip(lens, new)])
        q = _turn(s["qkv"][:, : c["n_q"]], freqs, pos, c, c["magnitude"])
        k = _turn(s["qkv"][:, c["n_q"]: c["n_q"] + n_kv], freqs, pos, c, c["magnitude"])
        v = s["qkv"][:, c["n_q"] + n_kv:].double()
        u = units(seq[:, None], head[None], pos[:, None], n_kv, cap, s["blocks"])
        row = (pos % 16)[:, None].expand(u.shape)
        return {"q": q, "k": _in_cache(_held(k, c["k"]), u, row, 0, n_units),
                "v": _in_cache(_held(v, c["v"]), u, row, 1, n_units), "lens": None}
    if op == "shift":
        into = s["k"].view(torch.float16).double() if c["k"] == F16 else None
        for i, (n, e) in enumerate(zip(lengths(c), evicted(c))):
            left = np.delete(np.arange(n), s["evict"][i, :e].cpu().numpy())
            w = torch.arange(n - e, device="cuda")
            u = units(torch.full_like(w, i)[:, None], head[None], w[:, None], n_kv, cap, s["blocks"])
            row = (w % 16)[:, None].expand(u.shape)
            by = w - torch.from_numpy(left).cuda()
            x = _read(s["k"], c["k"], 0, u, row)
            turned = _held(_turn(x, freqs, by, c), c["k"])
            into = _in_cache(torch.where((by != 0)[:, None, None], turned, x), u, row, 0, n_units, into)
        return {"k": into, "delta": None}
    lens = torch.tensor(lengths(c), device="cuda")
    q = _turn(s["q"], freqs, lens, c, c["magnitude"]).to(torch.float16).double()  # a query is fp16
    rows = [_held(_turn(s["k_new"], freqs, lens, c, c["magnitude"]), c["k"]), _held(s["v_new"].double(), c["v"])]
    got = {"out": [], "lse": []}
    back = [s[x].view(torch.float16).double() if c[x] == F16 else None for x in "kv"]
    for i, n in enumerate(lengths(c)):
        t = torch.arange(n + 1, device="cuda")
        u = units(torch.full_like(t, i)[:, None], head[None], t[:, None], n_kv, cap, s["blocks"])
        row = (t % 16)[:, None].expand(u.shape)
        sides = [_read(s[x], c[x], j, u, row) for j, x in enumerate("kv")]
        for j, x in enumerate("kv"):
            sides[j][n] = rows[j][i].to(torch.float16).double() if c[x] == F16 else rows[j][i]
            # f16 sides come back whole, others as the page that the step wrote to
            first = n if c[x] == F16 else n // 256 * 256
            back[j] = _in_cache(sides[j][first:], u[first:], row[first:], j, n_units, back[j])
        a = torch.einsum("hgd,thd->hgt", q[i].view(n_kv, -1, D), sides[0]) / math.sqrt(D)
        got["lse"].append(torch.logsumexp(a, -1).view(-1))
        got["out"].append(torch.einsum("hgt,thd->hgd", torch.softmax(a, -1), sides[1]).reshape(-1, D))
    return {"out": torch.stack(got["out"]), "lse": torch.stack(got["lse"]), "lens": None, "k": back[0], "v": back[1]}
