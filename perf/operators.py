"""The serving step around the compressed cache, as measured calls: rotary positions (tq_rope), appending rotated keys
and values to a paged cache (tq_append_kv, read back with tq_read_kv) and attention of ragged chunks of new tokens over
it (tq_chunk_attention).  `own` chooses between the plain form in torch operations and the library's calls."""
import functools
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
V_BITS = {"q8_0": 0, "turbo2_mse": 1, "turbo3_mse": 2, "turbo4_mse": 3}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of one sequence: the queries of a layer (32 heads of 128), far into a long context
        rope_case("rope-token", tokens=1, heads=32, d=128, rotary=128, layout="half", scaling="wavelength",
                  dtype="fp16", inverse=False, far=131072),
        # a prefill chunk's queries, bf16, stretched context
        rope_case("rope-chunk-4096", tokens=4096, heads=32, d=128, rotary=128, layout="half", scaling="yarn",
                  dtype="bf16", inverse=False, far=131072),
        # the gradient of partly rotated, interleaved 256-wide heads in fp32
        rope_case("rope-gradient-partial", tokens=2000, heads=16, d=256, rotary=64, layout="interleaved",
                  scaling="none", dtype="fp32", inverse=True, far=8192),
        # a decode batch: 64 sequences append one token each to 16-token pages
        append_case("append-decode-64", seqs=64, tokens=1, heads=8, d=128, page=16, dtype="fp16", v="q8_0",
                    rotary=128, layout="half", ctx=16384, mix=1),
        # one 4096-token chunk of the benchmark's model shape
        append_case("append-chunk-4096", seqs=1, tokens=4096, heads=8, d=128, page=64, dtype="bf16", v="q8_0",
                    rotary=128, layout="half", ctx=32768, mix=2),
        # a ragged batch of odd lengths, narrow heads, turbo V
        append_case("append-ragged-turbo-v", seqs=37, tokens=181, heads=8, d=64, page=16, dtype="fp16",
                    v="turbo3_mse", rotary=32, layout="interleaved", ctx=4096, mix=3),
        # latency: one token of one sequence at 32K context
        attend_case("attend-token-32k", seqs=1, tokens=1, heads=8, group=4, d=128, page=16, dtype="fp16", v="q8_0",
                    ctx=32768, mix=4),
        # a decode batch of 64 sequences of 1K to 16K tokens in shuffled 16-token pages
        attend_case("attend-decode-64", seqs=64, tokens=1, heads=8, group=4, d=128, page=16, dtype="fp16", v="q8_0",
                    ctx=16384, mix=5),
        # a prefill chunk deep in the context: the largest
        attend_case("attend-chunk-4096", seqs=1, tokens=4096, heads=8, group=4, d=128, page=64, dtype="bf16",
                    v="q8_0", ctx=32768, mix=6),
        # the asymmetric recipe (q8_0 K, 1-bit V, 4 KV heads of 8 query heads): a 512-token chunk at 32K
        attend_case("attend-asymmetric-512", seqs=1, tokens=512, heads=4, group=8, d=128, page=32, dtype="fp16",
                    v="turbo2_mse", ctx=32768, mix=7),
        # mixed prefill and decode, wide heads, capped scores and a sliding window
        attend_case("attend-capped-window", seqs=8, tokens=700, heads=4, group=2, d=256, page=64, dtype="bf16",
                    v="q8_0", ctx=8192, softcap=50.0, window=1024, mix=8),
        # packed documents behind a shared prefix with a distance bias, narrow heads, odd sizes
        attend_case("attend-documents-bias", seqs=5, tokens=333, heads=12, group=1, d=64, page=16, dtype="fp16",
                    v="turbo4_mse", ctx=2100, bias=True, documents=True, prefix=70, mix=9),
    ]


def rope_case(name, **k):
    return {"name": name, "op": "rope", **k}


def append_case(name, **k):
    return {"name": name, "op": "append", **k}


def attend_case(name, softcap=0.0, window=0, bias=False, documents=False, prefix=0, **k):
    return {"name": name, "op": "attend", "softcap": softcap, "window": window, "bias": bias, "documents": documents,
            "prefix": prefix, **k}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    d = rng.choice([64, 128, 256])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "rope":
        c = rope_case("", tokens=_log(rng, 1, 6000), heads=_log(rng, 1, 40), d=d,
                      rotary=rng.choice([d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                      layout=rng.choice(["half", "interleaved"]),
                      scaling=rng.choice(["none", "linear", "wavelength", "yarn"]),
                      dtype=rng.choice(["fp32", "fp16", "bf16"]), inverse=rng.random() < 0.3,
                      far=_log(rng, 1000, 1000000))
    elif op == "append":
        seqs = _log(rng, 1, 64)
        tokens = _log(rng, 1, 4096 // seqs)
        c = append_case("", seqs=seqs, tokens=tokens, heads=rng.randint(1, 10), d=d,
                        page=rng.choice([1, 16, 24, 64, 256]), dtype=rng.choice(["fp32", "fp16", "bf16"]),
                        v=rng.choice(list(V_BITS)), rotary=rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)]),
                        layout=rng.choice(["half", "interleaved"]), ctx=_log(rng, tokens, 16384),
                        mix=rng.randint(0, 1 << 30))
    else:
        seqs = _log(rng, 1, 48)
        tokens = rng.choice([1, _log(rng, 1, 1024 // seqs)])
        ctx = _log(rng, max(tokens, 16), min(32768, 400000 // seqs))
        c = attend_case("", seqs=seqs, tokens=tokens, heads=rng.choice([1, 2, 4, 5, 8]),
                        group=rng.choice([1, 2, 4, 7, 8]), d=d, page=rng.choice([16, 24, 64, 256]), dtype=dtype,
                        v=rng.choice(list(V_BITS)), ctx=ctx, softcap=rng.choice([0.0, 0.0, 30.0]),
                        window=rng.choice([0, 0, _log(rng, 10, 4096)]), bias=rng.random() < 0.3,
                        documents=rng.random() < 0.3, prefix=rng.choice([0, 0, _log(rng, 1, 500)]),
                        mix=rng.randint(0, 1 << 30))
    del c["name"]
    return c


def lengths(c):
    """New tokens and total length of each sequence: one of full size, the others anything down to one token."""
    r = random.Random(c["mix"])
    new = [c["tokens"]] + [_log(r, 1, c["tokens"]) for _ in range(c["seqs"] - 1)]
    total = [c["ctx"]] + [max(n, _log(r, max(1, c["ctx"] // 16), c["ctx"])) for n in new[1:]]
    return np.array(new, np.int64), np.array(total, np.int64)


def token_ranges(c):
    """Of every new token: its sequence, its position and the keys [lo, hi) it attends to."""
    new, total = lengths(c)
    seq = np.repeat(np.arange(len(new)), new)
    start = np.concatenate([[0], np.cumsum(new)[:-1]])
    pos = total[seq] - new[seq] + np.arange(len(seq)) - start[seq]
    prefix = np.minimum(total, c["prefix"])
    hi = np.minimum(total[seq], np.maximum(pos + 1, prefix[seq]))
    lo = np.maximum(0, pos - c["window"] + 1) if c["window"] else np.zeros_like(pos)
    first = np.zeros_like(pos)
    if c["documents"]:  # a document begins every 97 positions; every 50th token is padding and sees nothing
        first = pos // 97 * 97
        first[49::50] = total[seq][49::50]
        lo = np.maximum(lo, first)
    return seq, pos, lo, hi, first


def vector_bytes(v, d):
    return d + d // 16 if v == "q8_0" else d * V_BITS[v] // 8 + 2


def work(c):
    e = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["d"]
        return {"bytes": 2 * n * e + 4 * c["tokens"], "flops": 6 * c["tokens"] * c["heads"] * c["rotary"] // 2}
    if c["op"] == "append":  # k and v read, the cache written; then the rows read and written out in 16 bits
        n = int(lengths(c)[0].sum()) * c["heads"]
        stored = vector_bytes("q8_0", c["d"]) + vector_bytes(c["v"], c["d"])
        return {"bytes": n * (2 * c["d"] * e + 2 * stored + 4 * c["d"]), "flops": 20 * n * c["d"]}
    seq, pos, lo, hi, _ = token_ranges(c)
    some = hi > lo
    keys = sum(int(hi[some & (seq == b)].max() - lo[some & (seq == b)].min()) for b in np.unique(seq[some]))
    stored = vector_bytes("q8_0", c["d"]) + vector_bytes(c["v"], c["d"])
    hq = c["heads"] * c["group"]
    return {"bytes": keys * c["heads"] * stored + 2 * len(seq) * hq * c["d"] * e,
            "flops": 4 * c["d"] * hq * int(np.maximum(hi - lo, 0).sum())}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def normal(shape, seed, outliers=0.0):
    """N(0, 1) with a share of the last axis' channels 20 times larger, as cached keys and values have them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:
        n = shape[-1] * shape[-2]
        ch = torch.randperm(n, generator=g, device="cuda")[:max(1, int(outliers * n))]
        x.view(-1, n)[:, ch] *= 20
    return x


def pages(c, seed):
    """A shuffled block table of the sequences' pages, some pages left over."""
    _, total = lengths(c)
    blocks = -(-total // c["page"])
    rng = np.random.default_rng(seed)
    perm = rng.permutation(int(blocks.sum()) + 3).astype(np.int32)
    table = np.full((len(blocks), int(blocks.max())), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), int(blocks.sum()) + 3


def batch_state(c, seed):
    new, total = lengths(c)
    table, n_pages = pages(c, seed)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.repeat(np.arange(len(new)), new)
    return {"case": c, "table": table, "n_pages": n_pages, "cu": torch.from_numpy(cu).cuda(),
            "seq_lens": torch.from_numpy(total.astype(np.int32)).cuda(), "n_tokens": int(new.sum()),
            "seq_of": torch.from_numpy(seq).cuda(), "index_of": torch.from_numpy(np.arange(len(seq)) - cu[seq]).cuda(),
            "max_tokens": int(new.max()), "max_ctx": int(total.max())}


def prepare(case, seed):
    c = dict(case)
    if c["op"] == "rope":
        g = np.random.default_rng(seed)
        x = normal((c["tokens"], c["heads"], c["d"]), seed).to(DTYPES[c["dtype"]])
        pos = torch.from_numpy(g.integers(0, c["far"], c["tokens"]).astype(np.int32)).cuda()
        return {"case": c, "x": x, "positions": pos, "out": torch.empty_like(x)}
    s = batch_state(c, seed)
    H, d, P, n = c["heads"], c["d"], c["page"], s["n_tokens"]
    vectors = s["n_pages"] * H * P
    if c["op"] == "append":  # k and v of a fused projection, as its output has them: columns of one matrix
        qkv = normal((n, 4 * H, d), seed, 0.01).to(DTYPES[c["dtype"]])
        s |= {"qkv": qkv, "k": qkv[:, 2 * H:3 * H], "v": qkv[:, 3 * H:],
              "k_payload": torch.zeros(vectors * d, dtype=torch.uint8, device="cuda"),
              "k_header": torch.zeros(vectors * (d // 16), dtype=torch.uint8, device="cuda"),
              "k_out": torch.empty((n, H, d), dtype=torch.float16, device="cuda"),
              "v_out": torch.empty((n, H, d), dtype=torch.float16, device="cuda")}
        vb = vector_bytes(c["v"], d)
        head = d // 16 if c["v"] == "q8_0" else 2
        s["v_payload"] = torch.zeros(vectors * (vb - head), dtype=torch.uint8, device="cuda")
        s["v_header"] = torch.zeros(vectors * head, dtype=torch.uint8, device="cuda")
        return s
    s["q"] = normal((n, H * c["group"], d), seed + 7).to(DTYPES[c["dtype"]])
    s["out"] = torch.empty_like(s["q"])
    s["k_payload"], s["k_header"] = q8_cache(normal((s["n_pages"], P, H, d), seed + 1, 0.01))
    if c["v"] == "q8_0":
        s["v_payload"], s["v_header"] = q8_cache(normal((s["n_pages"], P, H, d), seed + 2, 0.01))
    else:
        s["v_payload"], s["v_header"] = turbo_cache(s["n_pages"], P, H, d, V_BITS[c["v"]], seed + 2)
    _, _, _, _, first = token_ranges(c)
    s["first"] = torch.from_numpy(first.astype(np.int32)).cuda() if c["documents"] else None
    s["prefix"] = torch.full((c["seqs"],), c["prefix"], dtype=torch.int32, device="cuda") if c["prefix"] else None
    hq = H * c["group"]
    s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda").float() / hq)) if c["bias"] else None
    return s


def q8_cache(x):
    """[pages, P, H, d] -> payload and header bytes in the cache's order [pages, H, P, ...]."""
    b = x.transpose(1, 2).reshape(*x.shape[:1], x.shape[2], x.shape[1], -1, 32)
    delta = b.abs().amax(-1, keepdim=True) / 127
    q = torch.clamp(torch.round(b / delta), -127, 127).to(torch.int8)
    return q.reshape(-1).view(torch.uint8), delta.half().reshape(-1).view(torch.uint8)


def turbo_cache(n_pages, P, H, d, bits, seed):
    """Codes of rotated Gaussian vectors, packed little-endian, and their norms."""
    y = normal((n_pages, H, P, d), seed)
    idx = torch.bucketize(y, torch.from_numpy(codebook(bits)[1]).float().cuda(), right=True)
    b = ((idx.unsqueeze(-1) >> torch.arange(bits, device="cuda")) & 1).reshape(-1, 8)
    payload = (b << torch.arange(8, device="cuda")).sum(-1).to(torch.uint8)
    norms = (math.sqrt(d) * (1 + 0.2 * torch.rand((n_pages, H, P), device="cuda",
                                                 generator=torch.Generator(device="cuda").manual_seed(seed + 5))))
    return payload, norms.half().reshape(-1).view(torch.uint8)


@functools.lru_cache(None)
def codebook(bits):
    """Lloyd-Max levels and borders of N(0, 1) with 2^bits levels (fp64)."""
    pdf = lambda t: math.exp(-0.5 * t * t) / math.sqrt(2 * math.pi) if math.isfinite(t) else 0.0  # noqa: E731
    cdf = lambda t: 0.5 * math.erfc(-t / math.sqrt(2))  # noqa: E731
    n = 1 << bits
    c = [-1.5 + 3.0 * (k + 0.5) / n for k in range(n)]
    for _ in range(5000):
        b = [-math.inf] + [0.5 * (c[k] + c[k + 1]) for k in range(n - 1)] + [math.inf]
        c = [(pdf(b[k]) - pdf(b[k + 1])) / (cdf(b[k + 1]) - cdf(b[k])) for k in range(n)]
        c = [0.5 * (c[k] - c[n - 1 - k]) for k in range(n)]
    return np.array(c), np.array([0.5 * (c[k] + c[k + 1]) for k in range(n - 1)])


@functools.lru_cache(None)
def signs(d):
    """The cache's sign diagonal of seed 1: the top bit of SplitMix64 at counters (1 << 32) + i."""
    z = (np.uint64(1 << 32) + np.arange(d, dtype=np.uint64)) + np.uint64(0x9E3779B97F4A7C15)
    z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
    z = z ^ (z >> np.uint64(31))
    return np.where((z >> np.uint64(63)) == 1, -1.0, 1.0)


@functools.lru_cache(None)
def rotation(d):
    """H diag(s), d x d, on the GPU in fp32."""
    h = np.array([[1.0]])
    while len(h) < d:
        h = np.block([[h, h], [h, -h]])
    return torch.from_numpy(h / math.sqrt(d) * signs(d)).float().cuda()


def rope_of(c):
    """The rotation's parameters: base 500000, stretched 8 times from 8192 tokens where a scaling is asked for."""
    return {"head_dim": c["d"], "rotary_dim": c["rotary"], "layout": c["layout"], "scaling": c.get("scaling", "none"),
            "base": 500000.0, "factor": 8.0, "original_ctx": 8192.0}


def frequencies(c):
    """Angles per position of the rotated pairs (fp64) and the factor on the rotated coordinates."""
    r, base, factor, orig = c["rotary"], 500000.0, 8.0, 8192.0
    i = np.arange(r // 2)
    f, scaling = base ** (-2.0 * i / r), c.get("scaling", "none")
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "wavelength":  # short waves as they are, long ones stretched, between 1 and 4 turns a blend
        s = np.clip((orig * f / (2 * math.pi) - 1.0) / 3.0, 0, 1)
        return f * s + f / factor * (1 - s), 1.0
    if scaling == "yarn":
        dim = lambda turns: r * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), r - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return run_own(s)
    if c["op"] == "rope":
        return plain_rope(s["x"].float(), s["positions"], c).to(s["x"].dtype)
    if c["op"] == "append":
        return plain_append(s)
    return plain_attend(s)


def plain_rope(x, positions, c):
    f, m = frequencies(c)
    r = c["rotary"]
    angle = positions.double()[:, None] * torch.from_numpy(f).cuda()
    cos, sin = (angle.cos() * m).float()[:, None], (angle.sin() * m).float()[:, None]
    if c.get("inverse"):
        sin = -sin
    x, rest = x[..., :r], x[..., r:]
    if c["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def plain_q8(x):
    b = x.reshape(*x.shape[:-1], -1, 32)
    delta = b.abs().amax(-1, keepdim=True) / 127
    t = torch.where(delta > 0, b / delta, 0.0)
    q = torch.sign(t) * torch.floor(t.abs() + 0.5)
    return (q * delta.half().float()).reshape(x.shape)


def plain_append(s):
    c = s["case"]
    pos = (s["seq_lens"].long() - (s["cu"][1:] - s["cu"][:-1]))[s["seq_of"]] + s["index_of"]
    k = plain_q8(plain_rope(s["k"].float(), pos, c))
    v = s["v"].float()
    if c["v"] == "q8_0":
        v = plain_q8(v)
    else:
        levels, borders = (torch.from_numpy(t).float().cuda() / math.sqrt(c["d"]) for t in codebook(V_BITS[c["v"]]))
        n = v.square().sum(-1, keepdim=True).sqrt()
        y = (v / torch.where(n > 0, n, 1.0)) @ rotation(c["d"]).T
        v = (n.half().float() * levels[torch.bucketize(y, borders, right=True)]) @ rotation(c["d"])
    page = s["table"].long()[s["seq_of"], pos // c["page"]]
    cache = torch.zeros((2, s["n_pages"], c["page"], c["heads"], c["d"]), dtype=torch.float16, device="cuda")
    cache[:, page, pos % c["page"]] = torch.stack([k, v]).half()
    return list(cache[:, page, pos % c["page"]])


def plain_values(payload, header, fmt, c, n_pages):
    """The stored values [pages, H, P, d] of a cache in fp32; turbo values still rotated."""
    shape = (n_pages, c["heads"], c["page"])
    if fmt == "q8_0":
        q = payload.view(torch.int8).view(*shape, -1, 32).float()
        return (q * header.view(torch.float16).view(*shape, -1, 1).float()).flatten(-2)
    bits = V_BITS[fmt]
    b = ((payload.unsqueeze(-1) >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1).view(-1, bits).int()
    idx = (b << torch.arange(bits, device="cuda", dtype=torch.int32)).sum(-1)
    levels = (torch.from_numpy(codebook(bits)[0]) / math.sqrt(c["d"])).float().cuda()
    return levels[idx].view(*shape, c["d"]) * header.view(torch.float16).view(*shape, 1).float()


def plain_attend(s):
    c = s["case"]
    B, H, G, d, n = c["seqs"], c["heads"], c["group"], c["d"], s["max_tokens"]
    table = s["table"].long().clamp(min=0)
    k, v = (plain_values(s[x + "_payload"], s[x + "_header"], f, c, s["n_pages"])[table]
            .transpose(1, 2).flatten(2, 3) for x, f in (("k", "q8_0"), ("v", c["v"])))
    T = k.shape[2]
    lens, new = s["seq_lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    i, j = torch.arange(n, device="cuda"), torch.arange(T, device="cuda")
    token = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["n_tokens"] - 1)
    pos = (lens - new)[:, None] + i  # [B, n]
    hi = pos + 1
    if s["prefix"] is not None:
        hi = torch.maximum(hi, s["prefix"].long()[:, None])
    lo = pos - c["window"] + 1 if c["window"] else torch.zeros_like(pos)
    if s["first"] is not None:
        lo = torch.maximum(lo, s["first"].long()[token])
    seen = (j >= lo[..., None]) & (j < torch.minimum(hi, lens[:, None])[..., None])  # [B, n, T]
    # a key after its sequence's end may hold anything: its value counts as zero
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    q = s["q"][token].float().view(B, n, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, d)
    score = (q @ k.transpose(-1, -2)).view(B, H, G, n, T) * (1 / math.sqrt(d))
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    if s["slopes"] is not None:
        far = (pos[..., None] - j).abs().float()
        score = score - s["slopes"].view(1, H, G, 1, 1) * far[:, None, None]
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    del score
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, H, G * n, T) @ v).view(B, H, G, n, d) / torch.where(total > 0, total, 1.0)
    if c["v"] != "q8_0":
        out = out @ rotation(d)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, H * G, d)
    return out[s["seq_of"], s["index_of"]].to(s["q"].dtype)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

@functools.lru_cache(None)
def context(d):
    from kv_cache_quantization_turbo_gb300 import tq
    return tq.tq_context_create(d, 1, 2)


def handles(s):
    """What a program keeps between its calls: views, the batch's description, the rotation, the workspace."""
    from kv_cache_quantization_turbo_gb300 import tq
    c = s["case"]
    h = {"tq": tq, "ctx": context(c["d"])}
    if c["op"] != "attend":
        h["rope"] = tq.tq_rope_build(**rope_of(c))
    if c["op"] != "rope":
        h["batch"] = tq.Batch(s["cu"], s["seq_lens"], s["table"], s["n_tokens"], s["max_tokens"], s["max_ctx"])
        h["k_view"], h["v_view"] = (tq.CacheView(f, c["d"], c["heads"], c["page"], s["n_pages"], 1, s[x + "_payload"],
                                                 s[x + "_header"]) for x, f in (("k", "q8_0"), ("v", c["v"])))
    if c["op"] == "attend":
        hq = c["heads"] * c["group"]
        h["scores"] = tq.ScoreMods(softcap=c["softcap"], window=c["window"], slopes=s["slopes"],
                                   first_keys=s["first"], prefix_lens=s["prefix"])
        h["bytes"] = tq.tq_chunk_workspace_bytes(h["ctx"], h["batch"], hq, c["heads"])
        h["workspace"] = torch.empty(h["bytes"], dtype=torch.uint8, device="cuda")
    s["handles"] = h
    return h


def run_own(s):
    c, h = s["case"], s.get("handles") or handles(s)
    tq, ctx, stream = h["tq"], h["ctx"], torch.cuda.current_stream()
    if c["op"] == "rope":
        status = tq.tq_rope(ctx, h["rope"], s["x"], s["positions"], s["out"], inverse=c["inverse"], stream=stream)
        out = s["out"]
    elif c["op"] == "append":
        status = tq.tq_append_kv(ctx, h["batch"], s["k"], s["v"], h["k_view"], h["v_view"], 0, rope=h["rope"],
                                 stream=stream)
        status = status or tq.tq_read_kv(ctx, h["batch"], h["k_view"], s["k_out"], h["v_view"], s["v_out"], 0,
                                         stream=stream)
        out = [s["k_out"], s["v_out"]]
    else:
        status = tq.tq_chunk_attention(ctx, h["batch"], s["q"], h["k_view"], h["v_view"], 0, 1 / math.sqrt(c["d"]),
                                       h["workspace"], h["bytes"], s["out"], mods=h["scores"], stream=stream)
        out = s["out"]
    if status:
        raise RuntimeError(tq.tq_status_string(status))
    return out


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact_rope(x, pos, c):
    """Pairs as complex numbers, turned by exp(i angle)."""
    f, m = frequencies(c)
    r = c["rotary"]
    turn = torch.polar(torch.full((len(pos), r // 2), m, dtype=torch.float64, device="cuda"),
                       pos.double()[:, None] * torch.from_numpy(f).cuda() * (-1.0 if c.get("inverse") else 1.0))
    y = x.double().clone()
    at = torch.arange(r // 2, device="cuda")
    first, second = (at, at + r // 2) if c["layout"] == "half" else (2 * at, 2 * at + 1)
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact_q8(x):
    out = torch.empty_like(x)
    for b in range(0, x.shape[-1], 32):
        part = x[..., b:b + 32]
        delta = part.abs().max(-1, keepdim=True).values / 127.0
        q = part / delta.clamp(min=1e-300)
        out[..., b:b + 32] = torch.trunc(q + 0.5 * torch.sign(q)) * delta.half().double()
    return out


def exact_rotate(x):
    """Orthonormal Walsh-Hadamard transform of the last axis by butterflies."""
    d, step = x.shape[-1], 1
    y = x
    while step < d:
        y = y.reshape(*x.shape[:-1], d // (2 * step), 2, step)
        y = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2)
        step *= 2
    return y.reshape(x.shape) / math.sqrt(d)


def exact_rows(payload, header, fmt, c, slots, head):
    """Stored vectors of one head at the given (page, offset) rows, in the original space."""
    page, off = slots
    d = c["d"]
    at = (page * c["heads"] + head) * c["page"] + off
    if fmt == "q8_0":
        q = payload.view(torch.int8).view(-1, d)[at].double()
        return q * header.view(torch.float16).view(-1, d // 32)[at].double().repeat_interleave(32, -1)
    bits = V_BITS[fmt]
    words = payload.view(-1, d * bits // 8)[at].int()
    codes = torch.zeros((len(at), d), dtype=torch.long, device="cuda")
    for bit in range(bits):
        n = torch.arange(d, device="cuda") * bits + bit
        codes |= ((words[:, n // 8] >> (n % 8)) & 1).long() << bit
    y = torch.from_numpy(codebook(bits)[0]).cuda()[codes] / math.sqrt(d)
    y = y * header.view(torch.float16)[at].double()[:, None]
    return exact_rotate(y) * torch.from_numpy(signs(d)).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return exact_rope(s["x"], s["positions"], c)
    new, total = lengths(c)
    if c["op"] == "append":
        pos = torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)]).cuda()
        k, v = exact_q8(exact_rope(s["k"], pos, c)), s["v"].double()
        if c["v"] == "q8_0":
            return [k, exact_q8(v)]
        levels, borders = (torch.from_numpy(t).cuda() / math.sqrt(c["d"]) for t in codebook(V_BITS[c["v"]]))
        sign = torch.from_numpy(signs(c["d"])).cuda()
        n = torch.linalg.vector_norm(v, dim=-1, keepdim=True)
        idx = torch.bucketize(exact_rotate(v * sign) / n.clamp(min=1e-300), borders, right=True)
        return [k, exact_rotate(levels[idx] * n.half().double()) * sign]
    _, pos, lo, hi, _ = token_ranges(c)
    pos, lo, hi = (torch.from_numpy(x).cuda() for x in (pos, lo, hi))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, t) in enumerate(zip(new.tolist(), total.tolist())):
        rows = slice(at, at + n)
        at += n
        j = torch.arange(t, device="cuda")
        slots = (s["table"][b].long()[j // c["page"]], j % c["page"])
        hidden = (j < lo[rows, None]) | (j >= hi[rows, None])
        empty = hidden.all(-1)
        for h in range(c["heads"]):
            k = exact_rows(s["k_payload"], s["k_header"], "q8_0", c, slots, h)
            v = exact_rows(s["v_payload"], s["v_header"], c["v"], c, slots, h)
            for g in range(h * c["group"], (h + 1) * c["group"]):
                z = s["q"][rows, g].double() @ k.T / math.sqrt(c["d"])
                if c["softcap"]:
                    z = c["softcap"] * torch.tanh(z / c["softcap"])
                if s["slopes"] is not None:
                    z = z - s["slopes"][g].double() * (pos[rows, None] - j).abs()
                z.masked_fill_(hidden, -math.inf)
                z[empty] = 0.0
                out[rows, g] = torch.where(empty[:, None], 0.0, torch.softmax(z, -1) @ v)
    return out
