"""Cases of the cached-scoring operators: per-head norm and rotation of queries
and keys with the cache write, slot maps of a paged key-value cache, causal
attention with a sliding window and sinks over packed sequences, and attention
of one new token over the paged cache.

``own`` false computes each operator from elementary torch operations in 32
bits (angles in 64); ``own`` true calls the library's entry points.  Every
length comes from the case itself (``lens`` seeds the ragged ones), every value
from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

ROT_BASE = 10000.0
NORM_EPS = 1e-6
HALF, INTERLEAVED = 0, 1


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a small batch: 16 heads of 128 (the 1.3B reward model's), latency
        {"name": "rope step 32", "op": "rope", "n": 32, "lo": 1, "hi": 1, "lens": 1, "far": 2048, "hq": 16,
         "hkv": 16, "d": 128, "rot": 128, "layout": HALF, "norm": True, "cache": "bf16", "page": 16},
        # its prompts: 64 sequences of 256-560 tokens, rotated once and written to the cache
        {"name": "rope prompts 64x256-560", "op": "rope", "n": 64, "lo": 256, "hi": 560, "lens": 2, "far": 0,
         "hq": 16, "hkv": 16, "d": 128, "rot": 128, "layout": HALF, "norm": True, "cache": "bf16", "page": 16},
        # grouped heads of 64, a quarter of each head rotated, far positions, an 8-bit cache
        {"name": "rope partial e4m3", "op": "rope", "n": 7, "lo": 301, "hi": 1777, "lens": 3, "far": 1000000,
         "hq": 12, "hkv": 4, "d": 64, "rot": 16, "layout": INTERLEAVED, "norm": False, "cache": "e4m3", "page": 64},
        # the step's slot map, and the one of a thousand short requests
        {"name": "slots step 64", "op": "slots", "n": 64, "lo": 1, "hi": 1, "lens": 4, "far": 4096, "page": 16},
        {"name": "slots prompts 1000x5-500", "op": "slots", "n": 1000, "lo": 5, "hi": 500, "lens": 5, "far": 0,
         "page": 16},
        # one request of 500 tokens: latency
        {"name": "decode 1x500", "op": "decode", "n": 1, "lo": 500, "hi": 500, "lens": 6, "hq": 12, "hkv": 12,
         "d": 64, "page": 16, "cache": "bf16", "window": 0, "sinks": 0},
        # the 1.3B shape's batch
        {"name": "decode 64x256-560", "op": "decode", "n": 64, "lo": 256, "hi": 560, "lens": 7, "hq": 16,
         "hkv": 16, "d": 128, "page": 16, "cache": "bf16", "window": 0, "sinks": 0},
        # a few long contexts beside short ones, grouped heads
        {"name": "decode 24x1-131071", "op": "decode", "n": 24, "lo": 1, "hi": 131071, "lens": 8, "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "cache": "bf16", "window": 0, "sinks": 0},
        # a wide batch with a window and sinks over an 8-bit cache
        {"name": "decode 128 window e4m3", "op": "decode", "n": 128, "lo": 100, "hi": 16384, "lens": 9, "hq": 32,
         "hkv": 8, "d": 128, "page": 32, "cache": "e4m3", "window": 4096, "sinks": 4},
        # short requests of the serving stream under a small window
        {"name": "window 64x2-100", "op": "window", "n": 64, "lo": 2, "hi": 100, "lens": 10, "hq": 12, "hkv": 12,
         "d": 64, "window": 32, "sinks": 4},
        # the 1.3B shape's prompts, every earlier token visible
        {"name": "window 64x256-560 all", "op": "window", "n": 64, "lo": 256, "hi": 560, "lens": 11, "hq": 16,
         "hkv": 16, "d": 128, "window": 0, "sinks": 0},
        # long documents under a window, grouped heads
        {"name": "window 5x1-32761", "op": "window", "n": 5, "lo": 1, "hi": 32761, "lens": 12, "hq": 32, "hkv": 8,
         "d": 128, "window": 4096, "sinks": 4},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lengths(n, lo, hi, seed):
    """n lengths in [lo, hi], spread evenly over their logarithm where the range is wide; the longest is hi."""
    r = random.Random(1000003 * seed + n)
    wide = hi > 100 * lo
    got = [_log_int(r, lo, hi) if wide else r.randint(lo, hi) for _ in range(n)]
    got[n // 2] = hi
    return np.array(got, dtype=np.int64)


def draw(rng):
    op = rng.choice(("rope", "slots", "decode", "window"))
    seed = rng.randrange(1, 1 << 30)
    page = rng.choice((8, 16, 24, 32, 64, 100, 128))
    hkv, group = rng.choice(((1, 8), (2, 5), (4, 3), (4, 8), (8, 4), (8, 1), (12, 1), (16, 1), (6, 2), (3, 16)))
    d = rng.choice((64, 128))
    cache = rng.choice(("bf16", "bf16", "e4m3"))
    if op == "rope":
        step = rng.random() < 0.4
        n = _log_int(rng, 1, 300) if step else _log_int(rng, 1, 64)
        lo, hi = (1, 1) if step else sorted((_log_int(rng, 2, 600), _log_int(rng, 2, 600)))
        return {"op": "rope", "n": n, "lo": lo, "hi": hi, "lens": seed, "far": rng.choice((0, 2048, 1000000)),
                "hq": hkv * group, "hkv": hkv, "d": d, "rot": rng.choice((d, d, d // 2, d // 4, 12, 36)),
                "layout": rng.choice((HALF, INTERLEAVED)), "norm": rng.random() < 0.6, "cache": cache, "page": page}
    if op == "slots":
        step = rng.random() < 0.4
        lo, hi = (1, 1) if step else sorted((_log_int(rng, 1, 700), _log_int(rng, 1, 700)))
        return {"op": "slots", "n": _log_int(rng, 1, 2000 if step else 700), "lo": lo, "hi": hi, "lens": seed,
                "far": rng.choice((0, 100, 5000)), "page": page}
    if op == "decode":
        n, top = _log_int(rng, 1, 256), _log_int(rng, 1, 131072)
        per = hkv * d * 4                                # bytes of one token's keys and values
        top = max(1, min(top, int(1.0e9 / (n * per))))
        lo = max(1, top // rng.choice((1, 3, 1000)))
        w = rng.random() < 0.4
        return {"op": "decode", "n": n, "lo": lo, "hi": top, "lens": seed, "hq": hkv * group, "hkv": hkv, "d": d,
                "page": page, "cache": cache, "window": _log_int(rng, 1, 5000) if w else 0,
                "sinks": rng.choice((0, 1, 4, 64)) if w else 0}
    w = rng.random() < 0.7
    top = _log_int(rng, 1, 12000 if w else 2000)
    n = _log_int(rng, 1, max(1, min(128, 24000 // top)))
    return {"op": "window", "n": n, "lo": max(1, top // rng.choice((1, 3, 200))), "hi": top, "lens": seed,
            "hq": hkv * group, "hkv": hkv, "d": d, "window": _log_int(rng, 1, 3000) if w else 0,
            "sinks": rng.choice((0, 1, 4, 64)) if w else 0}


def _visible(pos, window, sinks):
    """How many keys a query at each position of its sequence sees."""
    pos = np.asarray(pos, dtype=np.int64)
    if window <= 0:
        return pos + 1
    near = np.minimum(pos + 1, window)
    return near + np.minimum(np.maximum(pos + 1 - window, 0), sinks)


def work(case):
    lens = _lengths(case["n"], case["lo"], case["hi"], case["lens"])
    T, n = int(lens.sum()), case["n"]
    if case["op"] == "slots":
        pages = int((-(-lens // case["page"])).sum()) if not case["far"] else -(-T // case["page"])
        return {"bytes": 12 * n + 12 * T + 8 * pages + 16, "flops": T}
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "rope":
        item = 1 if case["cache"] == "e4m3" else 2
        per = (2 * hq + 3 * hkv) * d * 2 + 2 * hkv * d * item + 12        # q, k, v read; q, k and the cache written
        return {"bytes": T * per + case["rot"] * 4, "flops": T * (hq + hkv) * d * (8 if case["norm"] else 4)}
    if case["op"] == "decode":
        item = 1 if case["cache"] == "e4m3" else 2
        seen = int(_visible(lens - 1, case["window"], case["sinks"]).sum())
        pages = int((-(-lens // case["page"])).sum())
        return {"bytes": 2 * seen * hkv * d * item + 4 * n * hq * d + 4 * pages + 4 * n, "flops": 4 * seen * hq * d}
    seen = sum(int(_visible(np.arange(L), case["window"], case["sinks"]).sum()) for L in lens)
    return {"bytes": T * (2 * hq + 2 * hkv) * d * 2 + 4 * (n + 1), "flops": 4 * seen * hq * d}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _tables(before, new, page, seed, spare):
    """Block tables (pages in a shuffled order) for sequences of before + new tokens."""
    need = -(-(before + new) // page)
    total = int(need.sum()) + spare
    ids = np.random.RandomState(seed % (1 << 31)).permutation(total).astype(np.int32)
    width = max(1, int(need.max()))
    table = np.zeros((len(need), width), dtype=np.int32)
    ends = np.cumsum(need)
    for i, (e, k) in enumerate(zip(ends, need)):
        table[i, :k] = ids[e - k:e]
    return table, ids, need, total


def _cache(total, hkv, page, d, kind, g, filled):
    """Key and value pages [total][hkv][page][d]; e4m3 pages are held as bytes, with a scale for each head."""
    shape = (total, hkv, page, d)
    dev = g.device
    if kind == "bf16":
        if not filled:
            return torch.zeros(shape, dtype=torch.bfloat16, device=dev), \
                torch.zeros(shape, dtype=torch.bfloat16, device=dev), None, None
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g), \
            torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g), None, None
    ks = 0.02 + 0.03 * torch.rand(hkv, generator=g, device=dev)
    vs = 0.02 + 0.03 * torch.rand(hkv, generator=g, device=dev)
    if not filled:
        return torch.zeros(shape, dtype=torch.uint8, device=dev), torch.zeros(shape, dtype=torch.uint8, device=dev), ks, vs

    def fill(scale):
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        x /= scale.to(torch.bfloat16)[None, :, None, None]
        return x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    return fill(ks), fill(vs), ks, vs


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = np.random.RandomState(case["lens"])              # earlier lengths: the case's, as the lengths are
    lens = _lengths(case["n"], case["lo"], case["hi"], case["lens"])
    n, op = case["n"], case["op"]
    s = {"case": case}

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    if op == "slots":
        page = case["page"]
        before = r.randint(0, case["far"] + 1, n).astype(np.int64)
        table, ids, need, total = _tables(before, lens, page, seed, 32)
        held = -(-before // page)
        fresh = np.concatenate([ids[e - k:e][h:] for e, k, h in zip(np.cumsum(need), need, held)] + [ids[total - 32:]])
        np.random.RandomState(seed % (1 << 31)).shuffle(fresh)
        for i in range(n):
            table[i, held[i]:] = 0
        s.update(before=ints(before.astype(np.int32)), new=ints(lens.astype(np.int32)), table=ints(table), free=ints(fresh),
                 used=torch.full((1,), 3, dtype=torch.int32, device=dev), T=int(lens.sum()))
        s["out"] = {"offsets": torch.empty(n + 1, dtype=torch.int32, device=dev),
                    "positions": torch.empty(s["T"], dtype=torch.int32, device=dev),
                    "slots": torch.empty(s["T"], dtype=torch.int64, device=dev),
                    "length": torch.empty(n, dtype=torch.int32, device=dev),
                    "used": torch.empty(1, dtype=torch.int32, device=dev),
                    "unserved": torch.empty(1, dtype=torch.int32, device=dev)}
        return s

    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "rope":
        page, T = case["page"], int(lens.sum())
        first = r.randint(0, case["far"] + 1, n).astype(np.int64)
        held = first % page                              # the part of each sequence's last page that is taken
        table, _, _, total = _tables(held, lens, page, seed, 2)
        pos = np.concatenate([f + np.arange(L) for f, L in zip(first, lens)])
        at = np.concatenate([h + np.arange(L) for h, L in zip(held, lens)])
        seq = np.repeat(np.arange(n), lens)
        s["qkv"] = torch.empty(T, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        s["positions"] = ints(pos.astype(np.int32))
        s["slots"] = ints(table[seq, at // page].astype(np.int64) * page + at % page)
        s["freqs"] = ints(ROT_BASE ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"]))
        gain = lambda: 1 + 0.1 * torch.randn(d, generator=g, device=dev)  # noqa: E731
        s["q_gain"], s["k_gain"] = (gain(), gain()) if case["norm"] else (None, None)
        s["kc"], s["vc"], s["ks"], s["vs"] = _cache(total, hkv, page, d, case["cache"], g, False)
        s["q"] = torch.empty(T, hq * d, dtype=torch.bfloat16, device=dev)
        s["k"] = torch.empty(T, hkv * d, dtype=torch.bfloat16, device=dev)
        return s

    if op == "decode":
        table, _, _, total = _tables(np.zeros(n, dtype=np.int64), lens, case["page"], seed, 2)
        s["table"], s["length"] = ints(table), ints(lens.astype(np.int32))
        s["kc"], s["vc"], s["ks"], s["vs"] = _cache(total, hkv, case["page"], d, case["cache"], g, True)
        s["q"] = torch.empty(n, hq * d, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        s["o"] = torch.empty(n, hq * d, dtype=torch.bfloat16, device=dev)
        return s

    T = int(lens.sum())
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    s["offsets"], s["T"] = ints(off), T
    s["q"] = torch.empty(T, hq * d, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    s["k"] = torch.empty(T, hkv * d, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    s["v"] = torch.empty(T, hkv * d, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    s["o"] = torch.empty(T, hq * d, dtype=torch.bfloat16, device=dev)
    s["longest"] = int(lens.max())
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    return {"rope": _rope, "slots": _slots, "decode": _decode, "window": _window}[state["case"]["op"]](state)


def _handles(s):
    """The cache, rotation and workspace handles that a program keeps beside its buffers."""
    import classifier_scoring_b200 as rm

    c = s["case"]
    if "handle" not in s:
        if c["op"] in ("rope", "decode"):
            s["handle"] = rm.KvCache(s["kc"], s["vc"], n_pages=s["kc"].shape[0], page_size=c["page"], n_kv_heads=c["hkv"],
                                     head_dim=c["d"], dtype=rm.E4M3 if c["cache"] == "e4m3" else rm.BF16,
                                     k_scale=s["ks"], v_scale=s["vs"])
        if c["op"] == "rope":
            s["rope"] = rm.Rope(s["freqs"], c["rot"], layout=c["layout"])
        if c["op"] == "decode":
            size = rm.ops.attn_decode_workspace(c["n"], c["hq"], s["handle"])
            s["space"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
        s.setdefault("handle", None)
    return rm


def _slots(s):
    c, out = s["case"], s["out"]
    if own:
        rm = _handles(s)
        rm.ops.kv_slots(s["before"], s["new"], c["n"], c["page"], s["free"], s["free"].numel(), s["used"], s["table"],
                        s["table"].shape[1], s["T"], out["offsets"], out["positions"], out["slots"], out["length"],
                        out["used"], out["unserved"])
        return {**out, "table": s["table"]}
    before, new, table = s["before"].long(), s["new"].long(), s["table"]
    page, width = c["page"], table.shape[1]
    have = (before + page - 1) // page
    length = before + new
    want = (length + page - 1) // page - have
    pages = want.cumsum(0)
    ends = new.cumsum(0)
    fits = (pages <= s["free"].numel() - s["used"]) & (ends <= s["T"]) & (have + want <= width)
    served = fits.long().cumprod(0)
    new, want, length = new * served, want * served, before + new * served
    ends, pages = new.cumsum(0), want.cumsum(0)
    block = torch.arange(width, device=table.device)[None]
    fresh = (block >= have[:, None]) & (block < (have + want)[:, None])
    which = (s["used"].long() + (pages - want)[:, None] + block - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][which], table))
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(s["T"], device=table.device)
    seq = torch.searchsorted(ends, t, right=True).clamp_max(c["n"] - 1)
    at = before[seq] + t - offsets[seq]
    real = t < ends[-1]
    slot = table[seq, (at // page).clamp(0, width - 1)].long() * page + at % page
    return {"offsets": offsets.int(), "positions": torch.where(real, at, 0).int(), "slots": torch.where(real, slot, -1),
            "length": length.int(), "used": (s["used"] + pages[-1]).int(), "unserved": (c["n"] - served.sum()[None]).int(),
            "table": table}


def _rope(s):
    c = s["case"]
    T, hq, hkv, d, rot, page = s["qkv"].shape[0], c["hq"], c["hkv"], c["d"], c["rot"], c["page"]
    fp8 = c["cache"] == "e4m3"
    if own:
        rm = _handles(s)
        rm.ops.qk_norm_rope(s["qkv"], (hq + 2 * hkv) * d, s["q"], hq * d, s["k"], hkv * d, T, hq, hkv, d, s["q_gain"],
                            s["k_gain"], NORM_EPS, s["rope"], s["positions"], s["handle"], s["slots"])
    else:
        x = s["qkv"].view(T, hq + 2 * hkv, d).float()
        qk, v = x[:, :hq + hkv], x[:, hq + hkv:]
        if c["norm"]:
            qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + NORM_EPS)
            qk = torch.cat([qk[:, :hq] * s["q_gain"], qk[:, hq:] * s["k_gain"]], 1)
        angle = s["positions"].double()[:, None] * s["freqs"]
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        turn, rest = qk[..., :rot], qk[..., rot:]
        if c["layout"] == HALF:
            a, b = turn[..., :rot // 2], turn[..., rot // 2:]
            turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = turn[..., 0::2], turn[..., 1::2]
            turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        qk = torch.cat([turn, rest], -1)
        s["q"].copy_(qk[:, :hq].reshape(T, hq * d))
        s["k"].copy_(qk[:, hq:].reshape(T, hkv * d))
        at, row = s["slots"] // page, s["slots"] % page
        for buf, val, scale in ((s["kc"], qk[:, hq:], s["ks"]), (s["vc"], v, s["vs"])):
            if fp8:
                val = (val * (1 / scale)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            buf[at, :, row] = val.to(buf.dtype)
    see = (lambda b: b.view(torch.float8_e4m3fn)) if fp8 else (lambda b: b)
    return {"q": s["q"], "k": s["k"], "k_cache": see(s["kc"]), "v_cache": see(s["vc"])}


def _softmax_parts(score, seen):
    """exp(score - max) of the seen entries and their sum; a row that sees nothing gets zeros and the sum one."""
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    p = torch.where(seen, p, 0.0)
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, total, 1.0)


def _decode(s):
    c = s["case"]
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    if own:
        rm = _handles(s)
        rm.ops.attn_decode(s["q"], hq * d, s["handle"], s["table"], s["table"].shape[1], s["length"], n, hq, c["window"],
                           c["sinks"], s["o"], hq * d, s["space"])
        return s["o"]
    page, table = c["page"], s["table"].long()
    length = s["length"].long()[:, None]
    at = torch.arange(table.shape[1] * page, device=table.device)[None]
    seen = at < length
    if c["window"] > 0:
        seen = seen & ((at >= length - c["window"]) | (at < c["sinks"]))
    q = s["q"].view(n, hkv, hq // hkv, d).float()
    out = torch.empty(n, hkv, hq // hkv, d, device=q.device)
    for h in range(hkv):  # a key-value head at a time: the gathered pages in 32 bits are large
        k, v = (b[table, h].view(n, -1, d) for b in (s["kc"], s["vc"]))
        if c["cache"] == "e4m3":
            k, v = (b.view(torch.float8_e4m3fn).float() * w[h] for b, w in ((k, s["ks"]), (v, s["vs"])))
        score = torch.matmul(q[:, h], k.float().transpose(1, 2)) / math.sqrt(d)
        p, total = _softmax_parts(score, seen[:, None])
        out[:, h] = torch.matmul(p, v.float()) / total
    return out.view(n, hq * d).to(torch.bfloat16)


def _window(s):
    c = s["case"]
    T, n, hq, hkv, d = s["T"], c["n"], c["hq"], c["hkv"], c["d"]
    if own:
        rm = _handles(s)
        rm.ops.attn_window(s["q"], hq * d, s["k"], hkv * d, s["v"], hkv * d, s["offsets"], n, T, hq, hkv, d, c["window"],
                           c["sinks"], s["o"], hq * d)
        return s["o"]
    # blocks of 256 packed rows against the keys that any of them can see, and each row's sinks apart
    rows, dev = 256, s["q"].device
    w = c["window"] if c["window"] > 0 else s["longest"]
    w = min(w, s["longest"])
    blocks = -(-T // rows)
    row = torch.arange(blocks * rows, device=dev).view(blocks, rows)
    key = torch.arange(w + rows - 1, device=dev)[None] + (row[:, :1] - (w - 1))
    off = s["offsets"].long()
    start = off[(torch.searchsorted(off[1:].contiguous(), row, right=True)).clamp_max(n - 1)]
    inside, at = (key >= 0) & (key < T), key.clamp(0, T - 1)
    seen = inside[:, None] & (key[:, None] >= start[:, :, None]) & (key[:, None] <= row[:, :, None]) \
        & (key[:, None] > row[:, :, None] - w)
    first = start[:, :, None] + torch.arange(c["sinks"], device=dev)
    sunk = (first <= row[:, :, None] - w) & (row[:, :, None] < T)
    first, row = first.clamp(0, T - 1), row.clamp_max(T - 1)
    q, k, v = s["q"].view(T, hkv, hq // hkv, d), s["k"].view(T, hkv, d), s["v"].view(T, hkv, d)
    out = torch.empty(blocks * rows, hkv, hq // hkv, d, dtype=torch.bfloat16, device=dev)
    for h in range(hkv):  # a key-value head at a time: the scores in 32 bits are large
        qh = q[:, h][row].float().transpose(1, 2)                     # [blocks][group][rows][d]
        kh, vh = k[:, h][at].float()[:, None], v[:, h][at].float()[:, None]
        score = torch.cat([torch.matmul(qh, kh.transpose(2, 3)),
                           (qh[:, :, :, None] * k[:, h][first].float()[:, None]).sum(-1)], -1) / math.sqrt(d)
        p, total = _softmax_parts(score, torch.cat([seen, sunk], -1)[:, None])
        o = torch.matmul(p[..., :key.shape[1]], vh)
        o = o + (p[..., key.shape[1]:, None] * v[:, h][first].float()[:, None]).sum(-2)
        out[:, h] = (o / total).transpose(1, 2).reshape(blocks * rows, hq // hkv, d)
    return out.view(blocks * rows, hq * d)[:T]


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "slots":
        return None
    lens = _lengths(case["n"], case["lo"], case["hi"], case["lens"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    if op == "rope":
        T, rot = s["qkv"].shape[0], case["rot"]
        heads = s["qkv"].double().view(T, hq + 2 * hkv, d)[:, :hq + hkv].clone()
        if case["norm"]:
            heads /= (heads.pow(2).sum(-1, keepdim=True) / d + NORM_EPS).sqrt()
            heads[:, :hq] *= s["q_gain"].double()
            heads[:, hq:] *= s["k_gain"].double()
        z = torch.polar(torch.ones(1, dtype=torch.float64, device=heads.device),
                        s["positions"].double()[:, None] * s["freqs"])[:, None]
        i = torch.arange(rot // 2, device=heads.device)
        re, im = (i, i + rot // 2) if case["layout"] == HALF else (2 * i, 2 * i + 1)
        z = torch.complex(heads[:, :, re], heads[:, :, im]) * z
        heads[:, :, re], heads[:, :, im] = z.real, z.imag
        found = {"q": heads[:, :hq].reshape(T, hq * d), "k": heads[:, hq:].reshape(T, hkv * d), "k_cache": None, "v_cache": None}
        if case["cache"] == "bf16":                       # an 8-bit cache has its own grid of values
            flat = torch.zeros(s["kc"].shape[0] * case["page"], hkv, d, dtype=torch.float64, device=heads.device)
            flat[s["slots"]] = heads[:, hq:]
            found["k_cache"] = flat.view(-1, case["page"], hkv, d).transpose(1, 2).contiguous()
            flat = torch.zeros_like(flat)
            flat[s["slots"]] = s["qkv"].double().view(T, hq + 2 * hkv, d)[:, hq + hkv:]
            found["v_cache"] = flat.view(-1, case["page"], hkv, d).transpose(1, 2).contiguous()
        return found

    def attend(q, k, v, see):
        """q [hkv][rows][d], k and v [hkv][keys][d], see broadcast over [hkv][rows][keys]"""
        a = q @ k.transpose(1, 2) * d ** -0.5
        a = a.masked_fill(~see, -math.inf)
        return torch.softmax(a, -1) @ v

    if op == "decode":
        found = torch.zeros(case["n"], hq * d, dtype=torch.float64, device=s["q"].device)
        for i, L in enumerate(int(x) for x in lens):
            pages = s["table"][i, :-(-L // case["page"])].long()
            at = torch.arange(L, device=pages.device)
            if case["window"] > 0:
                at = at[(at >= L - case["window"]) | (at < case["sinks"])]
            kv = []
            for buf, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
                x = buf[pages[at // case["page"]], :, at % case["page"]]
                x = x.double() if scale is None else x.view(torch.float8_e4m3fn).double() * scale.double()[:, None]
                kv.append(x.transpose(0, 1))
            q = s["q"][i].double().view(hkv, group, d)
            found[i] = attend(q, *kv, torch.ones(1, dtype=torch.bool, device=q.device)).reshape(-1)
        return found
    found = torch.zeros(s["T"], hq * d, dtype=torch.float64, device=s["q"].device)
    b = 0
    for L in (int(x) for x in lens):
        for r0 in range(0, L, 1024):
            r1 = min(L, r0 + 1024)
            k0 = max(0, r0 - case["window"] + 1) if case["window"] > 0 else 0
            at = torch.arange(k0, r1, device=found.device)
            if k0 > 0 and case["sinks"] > 0:
                at = torch.cat([torch.arange(min(case["sinks"], k0), device=found.device), at])
            row = torch.arange(r0, r1, device=found.device).repeat(group)[:, None]
            see = at <= row
            if case["window"] > 0:
                see = see & ((at > row - case["window"]) | (at < case["sinks"]))
            for h in range(hkv):
                q = s["q"][b + r0:b + r1].view(-1, hkv, group, d)[:, h].double().transpose(0, 1).reshape(1, -1, d)
                k, v = (x[b + at].view(-1, hkv, d)[:, h].double()[None] for x in (s["k"], s["v"]))
                o = attend(q, k, v, see).view(group, r1 - r0, d).transpose(0, 1)
                found[b + r0:b + r1].view(-1, hkv, group, d)[:, h] = o
        b += L
    return found
