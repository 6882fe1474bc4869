"""Further operators of the serving step, as measured calls: norms of queries and keys per head with the rotation in the
same pass (tq_norm_rope) and their gradient (tq_norm_rope_grad); a cache in e4m3 with a scale for each block of 16 tokens
and head, written by tq_append_kv and read by tq_read_kv; ragged chunk attention over it, and over the q8_0 cache, with a
sliding window and first tokens that stay visible (tq_chunk_attention).  `own` chooses between the plain form in torch
operations and the library's calls."""
import functools
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 16   # tokens that share a scale
TOP = 448.0  # the largest e4m3 value
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of one sequence: the queries and keys of a layer (32 and 8 heads of 128), far into a context
        norm_case("norm-token", tokens=1, heads=32, kv_heads=8, d=128, rotary=128, layout="half", dtype="fp16",
                  far=131072),
        # a prefill chunk's queries and keys, as slices of a fused projection
        norm_case("norm-chunk-4096", tokens=4096, heads=32, kv_heads=8, d=128, rotary=128, layout="half", dtype="bf16",
                  far=131072),
        # a training step's gradient on the same rows
        norm_case("norm-gradient-4096", grad=True, tokens=4096, heads=32, kv_heads=8, d=128, rotary=128, layout="half",
                  dtype="bf16", far=131072),
        # wide heads, partly rotated, interleaved, in fp32, odd sizes
        norm_case("norm-gradient-partial", grad=True, tokens=777, heads=5, kv_heads=1, d=256, rotary=64,
                  layout="interleaved", dtype="fp32", far=8192),
        # a decode batch: 64 sequences append one token each to 16-token pages, next to up to 15 earlier tokens of a block
        append_case("append-decode-64", seqs=64, tokens=1, heads=8, d=128, page=16, dtype="fp16", rotary=128,
                    layout="half", ctx=16384, mix=1),
        # one 4096-token chunk of the benchmark's model shape
        append_case("append-chunk-4096", seqs=1, tokens=4096, heads=8, d=128, page=64, dtype="bf16", rotary=128,
                    layout="half", ctx=32768, mix=2),
        # a ragged batch of odd lengths, narrow heads, partly rotated
        append_case("append-ragged", seqs=37, tokens=181, heads=8, d=64, page=16, dtype="fp32", rotary=32,
                    layout="interleaved", ctx=4096, mix=3),
        # latency: one token of one sequence at 32K context
        attend_case("attend-token-32k", seqs=1, tokens=1, heads=8, group=4, d=128, page=16, dtype="fp16", ctx=32768,
                    mix=4),
        # a decode batch of 64 sequences of 1K to 16K tokens in shuffled 16-token pages
        attend_case("attend-decode-64", seqs=64, tokens=1, heads=8, group=4, d=128, page=16, dtype="fp16", ctx=16384,
                    mix=5),
        # a prefill chunk deep in the context: the largest
        attend_case("attend-chunk-4096", seqs=1, tokens=4096, heads=8, group=4, d=128, page=64, dtype="bf16", ctx=32768,
                    mix=6),
        # mixed prefill and decode, wide heads, a window with the first tokens kept
        attend_case("attend-window-sinks", seqs=8, tokens=700, heads=4, group=2, d=256, page=64, dtype="bf16", ctx=8192,
                    window=1024, sinks=16, mix=8),
        # a long-running decode batch over q8_0: a window and four first tokens
        attend_case("attend-window-sinks-q8", cache="q8_0", seqs=64, tokens=1, heads=8, group=4, d=128, page=16,
                    dtype="fp16", ctx=16384, window=4096, sinks=4, mix=9),
    ]


def norm_case(name, grad=False, **k):
    return {"name": name, "op": "norm", "grad": grad, **k}


def append_case(name, **k):
    return {"name": name, "op": "append", **k}


def attend_case(name, cache="f8_block", window=0, sinks=0, **k):
    return {"name": name, "op": "attend", "cache": cache, "window": window, "sinks": sinks, **k}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gradient", "append", "attend", "attend", "window"])
    d = rng.choice([64, 128, 256])
    rotary = rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)])
    layout = rng.choice(["half", "interleaved"])
    dtype = rng.choice(["fp16", "bf16"])
    if op in ("norm", "gradient"):
        c = norm_case("", grad=op == "gradient", tokens=_log(rng, 1, 5000), heads=_log(rng, 1, 40),
                      kv_heads=rng.randint(1, 8), d=d, rotary=rotary, layout=layout,
                      dtype=rng.choice(["fp32", "fp16", "bf16"]), far=_log(rng, 1000, 1000000))
    elif op == "append":
        seqs = _log(rng, 1, 64)
        tokens = _log(rng, 1, 4096 // seqs)
        c = append_case("", seqs=seqs, tokens=tokens, heads=rng.randint(1, 10), d=d, page=rng.choice([16, 48, 64, 256]),
                        dtype=rng.choice(["fp32", "fp16", "bf16"]), rotary=rotary, layout=layout,
                        ctx=_log(rng, tokens, 16384), mix=rng.randint(0, 1 << 30))
    else:
        seqs = _log(rng, 1, 48)
        tokens = rng.choice([1, _log(rng, 1, 1024 // seqs)])
        ctx = _log(rng, max(tokens, 16), min(32768, 400000 // seqs))
        kept = {"window": _log(rng, 10, 4096), "sinks": _log(rng, 1, 200)} if op == "window" else {}
        c = attend_case("", cache=rng.choice(["f8_block", "q8_0"]) if kept else "f8_block", seqs=seqs, tokens=tokens,
                        heads=rng.choice([1, 2, 4, 5, 8]), group=rng.choice([1, 2, 4, 7, 8]), d=d,
                        page=rng.choice([16, 48, 64, 256]), dtype=dtype, ctx=ctx, mix=rng.randint(0, 1 << 30), **kept)
    del c["name"]
    return c


def lengths(c):
    """New tokens and total length of each sequence: one of full size, the others anything down to one token."""
    r = random.Random(c["mix"])
    new = [c["tokens"]] + [_log(r, 1, c["tokens"]) for _ in range(c["seqs"] - 1)]
    total = [c["ctx"]] + [max(n, _log(r, max(1, c["ctx"] // 16), c["ctx"])) for n in new[1:]]
    return np.array(new, np.int64), np.array(total, np.int64)


def read_lengths(c):
    """Tokens of the blocks that an append touches: the new ones and those before them in their first block."""
    new, total = lengths(c)
    return total - (total - new) // BLOCK * BLOCK


def element(c):
    return 4 if c["dtype"] == "fp32" else 2


def vector_bytes(cache, d):
    """Stored bytes of a vector, its share of a block's scale among them."""
    return d + d // 16 if cache == "q8_0" else d + 4 / BLOCK


def work(c):
    e, d = element(c), c["d"]
    if c["op"] == "norm":
        n = c["tokens"] * (c["heads"] + c["kv_heads"]) * d
        if c["grad"]:  # x and the output's gradient read, the input's written
            return {"bytes": 3 * n * e + 4 * c["tokens"] + 2 * d * (e + 4), "flops": 16 * n}
        return {"bytes": 2 * n * e + 4 * c["tokens"] + 2 * d * e, "flops": 8 * n}
    if c["op"] == "append":  # k and v read, the cache written; then the touched blocks read and written out in 16 bits
        n, m = int(lengths(c)[0].sum()) * c["heads"], int(read_lengths(c).sum()) * c["heads"]
        stored = vector_bytes("f8_block", d)
        return {"bytes": int(n * (2 * d * e + 2 * stored) + m * (2 * stored + 4 * d)), "flops": 20 * n * d}
    new, total = lengths(c)
    keys = pairs = 0
    for n, t in zip(new.tolist(), total.tolist()):
        pos = np.arange(t - n, t)
        lo = np.maximum(pos - c["window"] + 1, 0) if c["window"] else np.zeros_like(pos)
        kept = np.minimum(lo, c["sinks"])
        pairs += int((pos + 1 - lo + kept).sum())
        keys += int(t - lo.min() + min(int(lo.min()), c["sinks"]))
    hq = c["heads"] * c["group"]
    return {"bytes": int(2 * keys * c["heads"] * vector_bytes(c["cache"], d) + 2 * int(new.sum()) * hq * d * e),
            "flops": 4 * d * hq * pairs}


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


def rows_of(new):
    """cu_tokens of a batch, and of every row its sequence and its index in it."""
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.repeat(np.arange(len(new)), new)
    return (torch.from_numpy(cu).cuda(), torch.from_numpy(seq).cuda(),
            torch.from_numpy(np.arange(len(seq)) - cu[seq]).cuda())


def prepare(case, seed):
    c = dict(case)
    d, t = c["d"], DTYPES[c["dtype"]]
    if c["op"] == "norm":  # q and k of a fused projection, as its output has them: columns of one matrix
        hq, hk, n = c["heads"], c["kv_heads"], c["tokens"]
        qkv = normal((n, hq + 2 * hk, d), seed, 0.01).to(t)
        pos = np.random.default_rng(seed).integers(0, c["far"], n).astype(np.int32)
        w = (1 + 0.2 * normal((2, d), seed + 1)).to(t)
        s = {"case": c, "qkv": qkv, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "wq": w[0], "wk": w[1],
             "positions": torch.from_numpy(pos).cuda(), "q_out": torch.empty((n, hq, d), dtype=t, device="cuda"),
             "k_out": torch.empty((n, hk, d), dtype=t, device="cuda")}
        if c["grad"]:
            s |= {"gq": normal((n, hq, d), seed + 2).to(t), "gk": normal((n, hk, d), seed + 3).to(t),
                  "dwq": torch.empty(d, device="cuda"), "dwk": torch.empty(d, device="cuda")}
        return s
    new, total = lengths(c)
    table, n_pages = pages(c, seed)
    cu, seq_of, index_of = rows_of(new)
    H, n = c["heads"], int(new.sum())
    s = {"case": c, "table": table, "n_pages": n_pages, "cu": cu, "seq_of": seq_of, "index_of": index_of,
         "seq_lens": torch.from_numpy(total.astype(np.int32)).cuda(), "n_tokens": n, "max_tokens": int(new.max()),
         "max_ctx": int(total.max())}
    store = f8_cache if c["op"] == "append" or c["cache"] == "f8_block" else q8_cache
    for i, x in enumerate("kv"):
        s[x + "_payload"], s[x + "_header"] = store(normal((n_pages, c["page"], H, d), seed + 1 + i, 0.01))
    if c["op"] == "append":
        qkv = normal((n, 4 * H, d), seed, 0.01).to(t)
        r = read_lengths(c)
        s["read_cu"], s["read_seq"], s["read_index"] = rows_of(r)
        m = int(r.sum())
        # the blocks that receive tokens, numbered in the order of the rows
        pos = np.concatenate([np.arange(b - a, b) for a, b in zip(new, total)])
        seq = np.repeat(np.arange(len(new)), new)
        first = np.concatenate([[True], (seq[1:] != seq[:-1]) | (pos[1:] // BLOCK != pos[:-1] // BLOCK)])
        s |= {"qkv": qkv, "k": qkv[:, 2 * H:3 * H], "v": qkv[:, 3 * H:], "read_tokens": m, "read_max": int(r.max()),
              "block_of": torch.from_numpy(np.cumsum(first) - 1).cuda(), "n_blocks": int(first.sum()),
              "k_out": torch.empty((m, H, d), dtype=torch.float16, device="cuda"),
              "v_out": torch.empty((m, H, d), dtype=torch.float16, device="cuda")}
        return s
    s["q"] = normal((n, H * c["group"], d), seed + 7).to(t)
    s["out"] = torch.empty_like(s["q"])
    return s


def q8_cache(x):
    """[pages, P, H, d] -> payload and header bytes in the cache's order [pages, H, P, ...]."""
    b = x.transpose(1, 2).reshape(*x.shape[:1], x.shape[2], x.shape[1], -1, 32)
    delta = b.abs().amax(-1, keepdim=True) / 127
    q = torch.clamp(torch.round(b / delta), -127, 127).to(torch.int8)
    return q.reshape(-1).view(torch.uint8), delta.half().reshape(-1).view(torch.uint8)


def scale_exponent(top):
    """The smallest e with top <= 448 2^e."""
    m, e = torch.frexp(top)
    return torch.where(top > 0, e - 9 + (m > 0.875).int(), -80).clamp(-80, 80)


def f8_cache(x):
    """[pages, P, H, d] -> e4m3 codes [pages, H, P, d] and a word for each block [pages, H, P / 16]: 2^e as fp32 bits."""
    b = x.transpose(1, 2).reshape(x.shape[0], x.shape[2], x.shape[1] // BLOCK, -1)
    e = scale_exponent(b.abs().amax(-1))
    code = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return code.reshape(-1).view(torch.uint8), ((e + 127) << 23).int().reshape(-1).view(torch.uint8)


def rope_of(c):
    return {"head_dim": c["d"], "rotary_dim": c["rotary"], "layout": c["layout"], "base": 500000.0}


def frequencies(c):
    """Angles per position of the rotated pairs (fp64)."""
    r = c["rotary"]
    return 500000.0 ** (-2.0 * np.arange(r // 2) / r)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return run_own(s)
    if c["op"] == "norm":
        return plain_gradient(s) if c["grad"] else plain_norm(s)
    if c["op"] == "append":
        return plain_append(s)
    return plain_attend(s)


def plain_rope(x, positions, c, inverse=False):
    r = c["rotary"]
    angle = positions.double()[:, None] * torch.from_numpy(frequencies(c)).cuda()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    x, rest = x[..., :r], x[..., r:]
    if c["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def plain_norm(s):
    c = s["case"]

    def part(x, w):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
        return plain_rope(y, s["positions"], c).to(x.dtype)
    return [part(s["q"], s["wq"]), part(s["k"], s["wk"])]


def plain_gradient(s):
    c = s["case"]

    def part(x, w, dy):
        y, g = x.float(), plain_rope(dy.float(), s["positions"], c, inverse=True)
        r = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        y = y * r
        gw = g * w.float()
        dx = r * (gw - y * (gw * y).mean(-1, keepdim=True))
        return dx.to(x.dtype), (g * y).double().sum((0, 1)).float()
    dq, dwq = part(s["q"], s["wq"], s["gq"])
    dk, dwk = part(s["k"], s["wk"], s["gk"])
    return [dq, dk, dwq, dwk]


def plain_append(s):
    c = s["case"]
    start = s["seq_lens"].long() - (s["cu"][1:] - s["cu"][:-1])
    pos = start[s["seq_of"]] + s["index_of"]
    page = s["table"].long()[s["seq_of"], pos // c["page"]]
    read_start = start // BLOCK * BLOCK
    at = read_start[s["read_seq"]] + s["read_index"]
    read_page = s["table"].long()[s["read_seq"], at // c["page"]]
    H, d, P = c["heads"], c["d"], c["page"]
    # a block keeps the scale of its earlier tokens, where it has some
    held = torch.zeros(s["n_blocks"], dtype=torch.bool, device="cuda")
    held.index_put_((s["block_of"],), (pos // BLOCK * BLOCK < start[s["seq_of"]]))
    outs = []
    for x, name in ((plain_rope(s["k"].float(), pos, c), "k"), (s["v"].float(), "v")):
        codes = s[name + "_payload"].view(torch.float8_e4m3fn).view(-1, H, P, d).float()
        e = (s[name + "_header"].view(torch.int32).view(-1, H, P // BLOCK) >> 23) - 127
        top = torch.zeros((s["n_blocks"], H), device="cuda").index_reduce_(0, s["block_of"], x.abs().amax(-1), "amax")
        now = scale_exponent(top)[s["block_of"]]
        before = e[page, :, pos % P // BLOCK]
        now = torch.where(held[s["block_of"]][:, None], torch.maximum(now, before), now)
        was, e = e, e.clone()
        e[page, :, pos % P // BLOCK] = now
        # earlier tokens take the block's scale too
        up = (was - e).float()
        old, new_e = codes[read_page, :, at % P], e[read_page, :, at % P // BLOCK]
        old = (old * torch.exp2(up[read_page, :, at % P // BLOCK])[..., None]).to(torch.float8_e4m3fn).float()
        new = torch.ldexp(x, -now.unsqueeze(-1)).to(torch.float8_e4m3fn).float()
        fresh = at >= start[s["read_seq"]]
        old[fresh] = new
        outs.append(torch.ldexp(old, new_e.unsqueeze(-1)).half())
    return outs


def plain_values(payload, header, c, n_pages):
    """The stored values [pages, H, P, d] of a cache in fp32."""
    shape = (n_pages, c["heads"], c["page"])
    if c["cache"] == "q8_0":
        q = payload.view(torch.int8).view(*shape, -1, 32).float()
        return (q * header.view(torch.float16).view(*shape, -1, 1).float()).flatten(-2)
    scale = header.view(torch.float32).view(n_pages, c["heads"], -1, 1, 1)
    code = payload.view(torch.float8_e4m3fn).view(n_pages, c["heads"], -1, BLOCK, c["d"]).float()
    return (code * scale).flatten(2, 3)


def plain_attend(s):
    c = s["case"]
    B, H, G, d, n = c["seqs"], c["heads"], c["group"], c["d"], s["max_tokens"]
    table = s["table"].long().clamp(min=0)
    k, v = (plain_values(s[x + "_payload"], s[x + "_header"], c, s["n_pages"])[table].transpose(1, 2).flatten(2, 3)
            for x in "kv")
    T = k.shape[2]
    lens, new = s["seq_lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    i, j = torch.arange(n, device="cuda"), torch.arange(T, device="cuda")
    token = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["n_tokens"] - 1)
    pos = (lens - new)[:, None] + i  # [B, n]
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])  # [B, n, T]
    if c["window"]:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    q = s["q"][token].float().view(B, n, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, d)
    score = (q @ k.transpose(-1, -2)).view(B, H, G, n, T) * (1 / math.sqrt(d))
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    del score
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, H, G * n, T) @ v).view(B, H, G, n, d) / torch.where(total > 0, total, 1.0)
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
    if c["op"] == "norm":
        if c["grad"]:
            h["bytes"] = tq.tq_norm_rope_grad_workspace_bytes(h["ctx"], c["tokens"], c["heads"] + c["kv_heads"])
    else:
        fmt = "f8_block" if c["op"] == "append" else c["cache"]
        h["batch"] = tq.Batch(s["cu"], s["seq_lens"], s["table"], s["n_tokens"], s["max_tokens"], s["max_ctx"])
        h["k_view"], h["v_view"] = (tq.CacheView(fmt, c["d"], c["heads"], c["page"], s["n_pages"], 1, s[x + "_payload"],
                                                 s[x + "_header"]) for x in "kv")
    if c["op"] == "append":
        h["read"] = tq.Batch(s["read_cu"], s["seq_lens"], s["table"], s["read_tokens"], s["read_max"], s["max_ctx"])
    if c["op"] == "attend":
        hq = c["heads"] * c["group"]
        h["scores"] = tq.ScoreMods(window=c["window"], sinks=c["sinks"])
        h["bytes"] = tq.tq_chunk_workspace_for(h["ctx"], h["batch"], hq, h["k_view"], h["v_view"], h["scores"])
    if "bytes" in h:
        h["workspace"] = torch.empty(h["bytes"], dtype=torch.uint8, device="cuda")
    s["handles"] = h
    return h


def run_own(s):
    c, h = s["case"], s.get("handles") or handles(s)
    tq, ctx, stream = h["tq"], h["ctx"], torch.cuda.current_stream()
    if c["op"] == "norm" and not c["grad"]:
        status = tq.tq_norm_rope(ctx, h["rope"], s["q"], s["q_out"], s["wq"], s["k"], s["k_out"], s["wk"], EPS,
                                 s["positions"], stream=stream)
        out = [s["q_out"], s["k_out"]]
    elif c["op"] == "norm":
        status = tq.tq_norm_rope_grad(ctx, h["rope"], s["q"], s["gq"], s["wq"], s["q_out"], s["dwq"], s["k"], s["gk"],
                                      s["wk"], s["k_out"], s["dwk"], EPS, s["positions"], h["workspace"], h["bytes"],
                                      stream=stream)
        out = [s["q_out"], s["k_out"], s["dwq"], s["dwk"]]
    elif c["op"] == "append":
        status = tq.tq_append_kv(ctx, h["batch"], s["k"], s["v"], h["k_view"], h["v_view"], 0, rope=h["rope"],
                                 stream=stream)
        status = status or tq.tq_read_kv(ctx, h["read"], h["k_view"], s["k_out"], h["v_view"], s["v_out"], 0,
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

def exact_rope(x, pos, c, sign=1.0):
    """Pairs as complex numbers, turned by exp(i angle)."""
    r = c["rotary"]
    angle = pos.double()[:, None] * torch.from_numpy(frequencies(c)).cuda() * sign
    turn = torch.polar(torch.ones_like(angle), angle)
    y = x.double().clone()
    at = torch.arange(r // 2, device="cuda")
    first, second = (at, at + r // 2) if c["layout"] == "half" else (2 * at, 2 * at + 1)
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact_norm(s):
    c, out, sums = s["case"], [], []
    for x, w, g in ((s["q"], s["wq"], "gq"), (s["k"], s["wk"], "gk")):
        x, w = x.double(), w.double()
        size = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["d"] + EPS)
        if not c["grad"]:
            out.append(exact_rope(x / size * w, s["positions"], c))
            continue
        dy = exact_rope(s[g], s["positions"], c, -1.0)
        sums.append((dy * x / size).sum((0, 1)))
        out.append(dy * w / size - x * (dy * x * w).sum(-1, keepdim=True) / (c["d"] * size ** 3))
    return out + sums


def exact_e4m3(x):
    """The nearest number of 4 significant bits, or multiple of 2^-9; a tie goes to the even one."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def exact_f8(payload, header, c, rows):
    """Codes and exponents of one cache at rows (page, offset): codes [n, H, d], exponents [n, H]."""
    page, off = rows
    H, P, d = c["heads"], c["page"], c["d"]
    vec = (page[:, None] * H + torch.arange(H, device="cuda")) * P + off[:, None]
    b = payload.view(-1, d)[vec].int()
    mant, ex = b & 7, (b >> 3) & 15
    value = torch.where(ex == 0, mant * 2.0 ** -9, (8 + mant) * torch.exp2(ex.double() - 10))
    word = header.view(torch.int32)[vec // BLOCK]
    return torch.where(b >= 128, -value, value), (word >> 23) - 127


def exact_append(s):
    c = s["case"]
    new, total = lengths(c)
    out = [[], []]
    at = 0
    for b, (n, t) in enumerate(zip(new.tolist(), total.tolist())):
        start = t - n
        pos = torch.arange(start // BLOCK * BLOCK, t, device="cuda")
        rows = (s["table"][b].long()[pos // c["page"]], pos % c["page"])
        old = start % BLOCK
        for i, x in enumerate((exact_rope(s["k"][at:at + n], pos[old:], c), s["v"][at:at + n].double())):
            code, e = exact_f8(s["kv"[i] + "_payload"], s["kv"[i] + "_header"], c, (rows[0][:old], rows[1][:old]))
            parts = []
            for j in range(0, len(pos), BLOCK):
                fresh = x[max(j - old, 0):j + BLOCK - old]
                top = fresh.abs().amax((0, 2))
                mant, ex = torch.frexp(top)
                now = torch.where(top > 0, ex - 9 + (mant > 0.875).int(), -80).clamp(-80, 80)
                if j < old:
                    now = torch.maximum(now, e[0])
                    parts.append(exact_e4m3(code * torch.exp2((e - now).double())[..., None])
                                 * torch.exp2(now.double())[:, None])
                scale = torch.exp2(now.double())[:, None]
                parts.append(exact_e4m3(fresh / scale) * scale)
            out[i].append(torch.cat(parts))
        at += n
    return [torch.cat(x) for x in out]


def exact_rows(s, x, rows, head):
    """Stored vectors of one head at (page, offset)."""
    c = s["case"]
    payload, header, d = s[x + "_payload"], s[x + "_header"], c["d"]
    if c["cache"] == "f8_block":
        one = dict(c, heads=1)
        code, e = exact_f8(payload, header, one, (rows[0] * c["heads"] + head, rows[1]))
        return (code * torch.exp2(e.double())[..., None])[:, 0]
    at = (rows[0] * c["heads"] + head) * c["page"] + rows[1]
    q = payload.view(torch.int8).view(-1, d)[at].double()
    return q * header.view(torch.float16).view(-1, d // 32)[at].double().repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "norm":
        return exact_norm(s)
    if c["op"] == "append":
        return exact_append(s)
    new, total = lengths(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, t) in enumerate(zip(new.tolist(), total.tolist())):
        rows = slice(at, at + n)
        at += n
        j, p = torch.arange(t, device="cuda"), torch.arange(t - n, t, device="cuda")[:, None]
        slots = (s["table"][b].long()[j // c["page"]], j % c["page"])
        hidden = j > p
        if c["window"]:
            hidden |= (p - j >= c["window"]) & (j >= c["sinks"])
        for h in range(c["heads"]):
            k, v = (exact_rows(s, x, slots, h) for x in "kv")
            for g in range(h * c["group"], (h + 1) * c["group"]):
                z = (s["q"][rows, g].double() @ k.T / math.sqrt(c["d"])).masked_fill_(hidden, -math.inf)
                out[rows, g] = torch.softmax(z, -1) @ v
    return out
