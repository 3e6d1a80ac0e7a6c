"""Cases and plain forms of the paged key/value cache's operators: rotary positions (`rope_apply`),
the cache write with its rotation and quantiser (`rope_kv_cache_append`, `kv_cache_append`), the
cache read-back (`kv_cache_gather`) and attention of single or tree-drafted tokens over the cache
(`attn_decode_paged`).

A case is a dict with "op" in {"rope", "append", "gather", "attend"}; its sequence lengths follow
from the case alone (a fixed low-discrepancy pattern), its contents and page order from the seed.
"""

import math
import random

import numpy as np
import torch

own = False

BASE = 10000.0
GOLDEN = 0.6180339887498949
DEV = "cuda"


def listed():
    return [
        # one decoding step's queries of a small model: launch latency
        dict(name="rope step", op="rope", tokens=7, heads=8, dim=64, rot=64, half=False, transpose=False,
             scaling="none", factor=1.0, max_pos=4096),
        # the queries of a training batch (2 x 8192 tokens, 16 heads of 128)
        dict(name="rope batch", op="rope", tokens=16384, heads=16, dim=128, rot=128, half=False, transpose=False,
             scaling="none", factor=1.0, max_pos=8192),
        # gradient through a part-rotated head whose positions were stretched to a long context
        dict(name="rope gradient, part of the head", op="rope", tokens=5003, heads=32, dim=256, rot=64, half=True,
             transpose=True, scaling="yarn", factor=16.0, max_pos=131072),
        # one decoding step of 16 sequences: rotate q and k, quantise k and v into their pages
        dict(name="append step e4m3", op="append", tokens=16, hq=32, hkv=8, dim=128, page=64, fp8=True,
             token_major=False, rope=True, rot=128, half=True, scaling="linear", factor=4.0, max_pos=32768, pad=0.0),
        # a prefill's keys and values written to the cache
        dict(name="append prefill e4m3", op="append", tokens=16384, hq=32, hkv=8, dim=128, page=128, fp8=True,
             token_major=False, rope=True, rot=128, half=False, scaling="none", factor=1.0, max_pos=16384, pad=0.0),
        # a ragged chunk with padded tokens into small token-major pages, without rotation
        dict(name="append chunk bf16", op="append", tokens=1777, hq=12, hkv=12, dim=64, page=16, fp8=False,
             token_major=True, rope=False, rot=64, half=False, scaling="none", factor=1.0, max_pos=4096, pad=0.07),
        # cached prefixes of nine requests read back for a prefill of their next chunks
        dict(name="gather prefixes e4m3", op="gather", seqs=9, longest=4096, ragged=0.9, hkv=16, dim=128, page=64,
             fp8=True, token_major=False),
        # three short prefixes in small pages
        dict(name="gather short bf16", op="gather", seqs=3, longest=517, ragged=0.95, hkv=8, dim=64, page=16,
             fp8=False, token_major=True),
        # one sequence, one new token: latency
        dict(name="decode one bf16", op="attend", batch=1, draft=1, hq=32, hkv=8, dim=128, page=16, longest=1000,
             ragged=0.0, fp8=False, token_major=False, tree=False),
        # a serving batch's step over a quantised cache
        dict(name="decode batch e4m3", op="attend", batch=16, draft=1, hq=32, hkv=8, dim=128, page=64, longest=8192,
             ragged=0.3, fp8=True, token_major=False, tree=False),
        # verification of a 32-token tree for every sequence (128 query rows per key/value head)
        dict(name="tree of 32 bf16", op="attend", batch=8, draft=32, hq=32, hkv=8, dim=128, page=128, longest=8192,
             ragged=0.5, fp8=False, token_major=False, tree=True),
        # small trees at long contexts, quantised cache
        dict(name="tree of 8 long e4m3", op="attend", batch=3, draft=8, hq=32, hkv=8, dim=128, page=64,
             longest=65536, ragged=0.6, fp8=True, token_major=False, tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "gather", "attend", "attend"])
    dim = rng.choice([64, 128, 256]) if op != "attend" else rng.choice([64, 128])
    half = rng.random() < 0.5
    scaling, factor = rng.choice([("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
    rot = rng.choice([dim, dim // 2, dim // 4])
    page = rng.choice([16, 32, 64, 128, 256])
    fp8, token_major = rng.random() < 0.6, rng.random() < 0.4
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "rope":
        heads = rng.choice([1, 3, 8, 16, 32])
        tokens = min(_log(rng, 1, 16384), 16384 * 2048 // (heads * dim))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, rot=rot, half=half, transpose=rng.random() < 0.5,
                    scaling=scaling, factor=factor, max_pos=_log(rng, 128, 131072))
    if op == "append":
        hq = hkv * rng.choice([1, 4, 7, 8]) if hkv <= 8 else hkv
        tokens = min(_log(rng, 1, 16384), 16384 * 6144 // ((hq + 2 * hkv) * dim))
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, dim=dim, page=page, fp8=fp8, token_major=token_major,
                    rope=rng.random() < 0.7, rot=rot, half=half, scaling=scaling, factor=factor,
                    max_pos=_log(rng, 128, 131072), pad=rng.choice([0.0, 0.1]))
    if op == "gather":
        seqs = _log(rng, 1, 64)
        longest = max(1, min(_log(rng, 1, 16384), 9 * 4096 * 2048 // (seqs * hkv * dim)))
        return dict(op=op, seqs=seqs, longest=longest, ragged=rng.uniform(0, 1), hkv=hkv, dim=dim, page=page,
                    fp8=fp8, token_major=token_major)
    draft = rng.choice([1, 1, 2, 5, 8, 16, 33, 64])
    group = rng.choice([1, 4, 7, 8])
    batch = _log(rng, 1, 64)
    most = min(65536, 16 * 8192 * 8 * 128 // (batch * hkv * dim), 8 * 32 * 32 * 8192 // (batch * hkv * group * draft))
    longest = _log(rng, 1, max(2, most))
    return dict(op=op, batch=batch, draft=draft, hq=hkv * group, hkv=hkv, dim=dim, page=page, longest=longest,
                ragged=rng.uniform(0, 1), fp8=fp8, token_major=token_major, tree=draft > 1 and rng.random() < 0.8)


# ---------------------------------------------------------------- inputs --

def _lengths(n, longest, ragged):
    """n lengths from longest * (1 - ragged) to longest, the first one longest."""
    return [max(0, longest - int(longest * ragged * ((i * GOLDEN) % 1.0))) for i in range(n)]


def _drafts(c):
    """Drafted tokens of each sequence: `draft`, for trees every third sequence two fewer."""
    return [c["draft"] - (2 if c["tree"] and c["draft"] > 2 and b % 3 == 2 else 0) for b in range(c["batch"])]


def _theta(rot, scaling, factor, length):
    """Frequencies (fp64) and the multiplier of cos and sin.  linear: positions divided by the
    factor; ntk: base * factor^(d / (d - 2)); yarn: by parts, by the turns a pair makes within the
    original length (below 1 as linear, above 32 unscaled), multiplier 0.1 ln(factor) + 1."""
    base = BASE
    if scaling == "ntk":
        base = BASE * factor ** (rot / (rot - 2))
    th = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        th = [t / factor for t in th]
    if scaling == "yarn":
        ramp = [min(1.0, max(0.0, (length * t / (2 * math.pi) - 1.0) / 31.0)) for t in th]
        th = [(1 - g) * t / factor + g * t for t, g in zip(th, ramp)]
    return th, (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def _original(c):
    return max(1, int(c["max_pos"] / c["factor"]))


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _rows_quantised(x):
    """E4M3 rows of x and their fp32 scales (largest magnitude / 448; 1 for a row of zeros)."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _cache(g, pages, hkv, page, dim, fp8, token_major):
    """A key/value cache that holds earlier tokens everywhere."""
    out = []
    for _ in range(2):
        x = _randn((pages, hkv, page, dim), g)
        if fp8:
            x, scale = _rows_quantised(x)
        else:
            x, scale = x.to(torch.bfloat16), None
        out.append((x.transpose(1, 2).contiguous() if token_major else x, scale))
    return out


def _table(g, lens, page):
    """A page table (int32, unused entries -1) for sequences of these lengths, pages in random
    order, and the number of pages of the cache (a few of them free)."""
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu().numpy()
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(table).to(DEV), pages


def _tree(c, drafts, seed):
    """Per drafted token the set of drafted tokens it sees (its ancestors and itself), as bits."""
    r = random.Random(seed)
    mask = np.zeros((c["batch"], c["draft"]), np.uint64)
    for b in range(c["batch"]):
        seen = []
        for t in range(drafts[b]):
            parent = r.randrange(max(0, t - 6) - 1, t)
            seen.append((seen[parent] if parent >= 0 else 0) | (1 << t))
        mask[b, :drafts[b]] = np.array(seen, np.uint64)
    return torch.from_numpy(mask.view(np.int64)).to(DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("rope", "append"):
        s["theta"], s["gain"] = _theta(c["rot"], c["scaling"], c["factor"], _original(c))
        s["theta"] = torch.tensor(s["theta"], dtype=torch.float64, device=DEV)
        first = int(torch.randint(0, max(1, c["max_pos"] - c["tokens"]) , (1,), generator=g, device=DEV).item())
        s["pos"] = ((torch.arange(c["tokens"], device=DEV) + first) % c["max_pos"]).to(torch.int32)
        if own:
            from exact_attention_46_gb300 import ops
            s["cs"] = ops.rope_scaled_table(c["max_pos"], c["rot"], BASE, c["scaling"], c["factor"], _original(c))
    if c["op"] == "rope":
        s["x"] = _randn((c["tokens"], c["heads"], c["dim"]), g).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["x"])
    elif c["op"] == "append":
        # q, k and v are views of one projection's output
        T, hq, hkv, D, P = c["tokens"], c["hq"], c["hkv"], c["dim"], c["page"]
        qkv = _randn((T, hq + 2 * hkv, D), g).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        pages = (T + P - 1) // P + 3
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _cache(g, pages, hkv, P, D, c["fp8"], c["token_major"])
        # consecutive tokens fill pages that lie anywhere; padded tokens have slot -1
        perm = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        slots = perm[t // P] * P + t % P
        s["slots"] = torch.where(torch.rand(T, generator=g, device=DEV) < c["pad"], -1, slots)
        s["q_out"] = torch.empty((T, hq, D), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "gather":
        lens = _lengths(c["seqs"], c["longest"], c["ragged"])
        s["table"], pages = _table(g, lens, c["page"])
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _cache(g, pages, c["hkv"], c["page"], c["dim"], c["fp8"], c["token_major"])
        s["total"] = sum(lens)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
        shape = (s["total"], c["hkv"], c["dim"])
        s["ko"], s["vo"] = (torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    else:
        drafts, ctx = _drafts(c), _lengths(c["batch"], c["longest"], c["ragged"])
        s["table"], pages = _table(g, [a + b for a, b in zip(ctx, drafts)], c["page"])
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _cache(g, pages, c["hkv"], c["page"], c["dim"], c["fp8"], c["token_major"])
        s["q"] = _randn((c["batch"], c["draft"], c["hq"], c["dim"]), g).to(torch.bfloat16)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        s["drafts"] = torch.tensor(drafts, dtype=torch.int32, device=DEV)
        s["mask"] = _tree(c, drafts, seed) if c["tree"] else None
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((c["batch"], c["hq"], c["draft"]), dtype=torch.float32, device=DEV)
        if own:
            from exact_attention_46_gb300 import ops
            need = ops.decode_paged_workspace_bytes(c["batch"], c["draft"], c["hq"], c["hkv"], c["dim"], c["page"],
                                                    s["table"].shape[1])
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------- plain forms --

def _rotate(x, pos, theta, gain, rot, half, transpose):
    """Rotary positions of x [T, H, D] in fp32 (the angles in 64 bits), not yet rounded."""
    ang = pos.double()[:, None] * theta
    cos, sin = (ang.cos() * gain).float()[:, None], (ang.sin() * gain).float()[:, None]
    if transpose:
        sin = -sin
    x = x.float()
    out = x.clone()
    if half:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    return out


def _plain_append(s):
    c = s["case"]
    k, v = s["k"].float(), s["v"].float()
    if c["rope"]:
        k = _rotate(s["k"], s["pos"], s["theta"], s["gain"], c["rot"], c["half"], False)
        s["q_out"].copy_(_rotate(s["q"], s["pos"], s["theta"], s["gain"], c["rot"], c["half"], False))
    keep = s["slots"] >= 0
    page, at = s["slots"][keep] // c["page"], s["slots"][keep] % c["page"]
    for x, cache, scales in ((k[keep], s["kc"], s["ks"]), (v[keep], s["vc"], s["vs"])):
        rows = cache if c["token_major"] else cache.transpose(1, 2)      # [pages, page, heads, dim]
        if c["fp8"]:
            amax = x.abs().amax(-1)
            scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
            scales.transpose(1, 2)[page, at] = scale
            x = (x.double() / scale.double()[..., None]).clamp(-448, 448).float().to(torch.float8_e4m3fn)
            rows.view(torch.uint8)[page, at] = x.view(torch.uint8)
        else:
            rows[page, at] = x.to(torch.bfloat16)


def _read(cache, scales, token_major, page, at):
    """fp32 rows [..., heads, dim] of the cache at (page, at)."""
    rows = cache if token_major else cache.transpose(1, 2)
    if scales is None:
        return rows[page, at].float()
    return rows.view(torch.uint8)[page, at].view(torch.float8_e4m3fn).float() * scales.transpose(1, 2)[page, at][..., None]


def _plain_gather(s):
    c = s["case"]
    t = torch.arange(s["total"], device=DEV)
    seq = (t[:, None] >= s["cu"][None, 1:]).sum(-1)
    off = t - s["cu"].long()[seq]
    page = s["table"].long()[seq, off // c["page"]]
    s["ko"].copy_(_read(s["kc"], s["ks"], c["token_major"], page, off % c["page"]))
    s["vo"].copy_(_read(s["vc"], s["vs"], c["token_major"], page, off % c["page"]))


def _plain_attend(s):
    c = s["case"]
    B, T, Hq, D = s["q"].shape
    G = Hq // c["hkv"]
    L = s["table"].shape[1] * c["page"]
    j = torch.arange(L, device=DEV)
    page = s["table"].long().clamp(min=0)[:, j // c["page"]]                         # [B, L]
    k = _read(s["kc"], s["ks"], c["token_major"], page, j % c["page"])               # [B, L, Hkv, D]
    v = _read(s["vc"], s["vs"], c["token_major"], page, j % c["page"])
    ctx, drafts = s["ctx"].long()[:, None, None], s["drafts"].long()[:, None, None]
    i, t = j[None, None] - ctx, torch.arange(T, device=DEV)[None, :, None]           # drafted key, drafted query
    if s["mask"] is None:
        sees = i <= t
    else:
        sees = ((s["mask"][:, :, None] >> i.clamp(0, 63)) & 1) == 1
    sees = (i < 0) | (sees & (i < drafts))                                            # [B, T, L]
    q = s["q"].float().reshape(B, T, c["hkv"], G, D)
    x = torch.einsum("btkgd,blkd->bkgtl", q, k) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bkgtl,blkd->btkgd", p / total.clamp(min=1e-38), v).reshape(B, T, Hq, D)
    lse = (m + torch.log(total)).reshape(B, Hq, T)
    real = (t < drafts)[:, :, 0]                                                      # [B, T]
    s["o"].copy_(torch.where(real[:, :, None, None], o.to(torch.bfloat16), s["o"]))
    s["lse"].copy_(torch.where(real[:, None], lse, s["lse"]))


def run(state):
    s = state
    c = s["case"]
    if own:
        from exact_attention_46_gb300 import ops
    if c["op"] == "rope":
        if own:
            ops.rope_apply(s["x"], s["cs"], s["pos"], half=c["half"], transpose=c["transpose"], out=s["out"])
        else:
            s["out"].copy_(_rotate(s["x"], s["pos"], s["theta"], s["gain"], c["rot"], c["half"], c["transpose"]))
        return {"x": s["out"]}
    if c["op"] == "append":
        if not own:
            _plain_append(s)
        elif c["rope"]:
            ops.rope_kv_cache_append(s["q"], s["k"], s["v"], s["cs"], s["pos"], s["kc"], s["vc"], s["slots"], s["ks"],
                                     s["vs"], half=c["half"], token_major=c["token_major"], q_out=s["q_out"])
        else:
            ops.kv_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["ks"], s["vs"],
                                token_major=c["token_major"])
        return {"k": s["kc"], "v": s["vc"], "ks": s["ks"], "vs": s["vs"], "q": s["q_out"] if c["rope"] else None}
    if c["op"] == "gather":
        if own:
            ops.kv_cache_gather(s["kc"], s["vc"], s["table"], s["cu"], s["total"], s["ks"], s["vs"],
                                token_major=c["token_major"], k_out=s["ko"], v_out=s["vo"])
        else:
            _plain_gather(s)
        return {"k": s["ko"], "v": s["vo"]}
    if own:
        ops.attn_decode_paged(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["ks"], s["vs"], q_lens=s["drafts"],
                              tree_mask=s["mask"], token_major=c["token_major"], out=s["o"], lse=s["lse"],
                              workspace=s["ws"])
    else:
        _plain_attend(s)
    return {"o": s["o"], "lse": s["lse"]}


# ---------------------------------------------------- work, exact values --

def work(case):
    c = case
    row = c["dim"] * (1 if c.get("fp8") else 2) + (4 if c.get("fp8") else 0)          # one cached head of one token
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 4 * n + 4 * c["tokens"], "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    if c["op"] == "append":
        T = c["tokens"]
        b = 2 * T * c["hkv"] * (2 * c["dim"] + row) + 8 * T
        f = 2 * T * c["hkv"] * c["dim"] * (2 if c["fp8"] else 0)
        if c["rope"]:
            b += 4 * T * c["hq"] * c["dim"] + 4 * T
            f += 3 * T * (c["hq"] + c["hkv"]) * c["rot"]
        return {"bytes": b, "flops": f}
    if c["op"] == "gather":
        n = sum(_lengths(c["seqs"], c["longest"], c["ragged"])) * c["hkv"]
        return {"bytes": 2 * n * (row + 2 * c["dim"]), "flops": 2 * n * c["dim"] if c["fp8"] else 0}
    drafts, ctx = _drafts(c), _lengths(c["batch"], c["longest"], c["ragged"])
    keys = sum(a + b for a, b in zip(ctx, drafts))
    rows = sum(drafts) * c["hq"]
    pairs = sum((a + b) * b for a, b in zip(ctx, drafts)) * c["hq"]
    return {"bytes": 2 * keys * c["hkv"] * row + rows * (4 * c["dim"] + 4), "flops": 4 * pairs * c["dim"]}


def _turned64(x, pos, theta, gain, rot, half, transpose):
    """x * exp(+-i pos theta) on complex pairs, in 64 bits."""
    z = x.double()
    lead = z[..., :rot]
    pairs = lead.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if half else lead.unflatten(-1, (rot // 2, 2))
    turn = torch.polar(torch.full_like(theta, gain).expand(len(pos), -1), pos.double()[:, None] * theta)
    if transpose:
        turn = turn.conj()
    w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    w = w.transpose(-1, -2).flatten(-2) if half else w.flatten(-2)
    return torch.cat([w, z[..., rot:]], -1)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "rope":
        return {"x": _turned64(s["x"], s["pos"], s["theta"], s["gain"], c["rot"], c["half"], c["transpose"])}
    if c["op"] == "append":
        turn = (s["pos"], s["theta"], s["gain"], c["rot"], c["half"], False)
        k, v = (_turned64(s["k"], *turn) if c["rope"] else s["k"].double()), s["v"].double()
        keep = torch.nonzero(s["slots"] >= 0).flatten()
        page = torch.div(s["slots"][keep], c["page"], rounding_mode="floor")
        at = s["slots"][keep] - page * c["page"]
        out = {"q": _turned64(s["q"], *turn) if c["rope"] else None, "ks": None, "vs": None}
        for name, x in (("k", k[keep]), ("v", v[keep])):
            cache = s[name + "c"].to(torch.float64)
            if c["fp8"]:
                scales = s[name + "s"].double()
                top = x.abs().max(-1).values / 448
                top = torch.where(top == 0, torch.ones_like(top), top)
                x = x / top[..., None]
                scales.movedim(1, 2)[page, at] = top
                out[name + "s"] = scales
            (cache if c["token_major"] else cache.movedim(1, 2))[page, at] = x
            out[name] = cache
        return out
    heads = c["hkv"]

    def rows(name, b, n):
        """[n, heads, dim] of sequence b's first n tokens in 64 bits."""
        pages = s["table"][b, :(n + c["page"] - 1) // c["page"]].long()
        x = s[name + "c"][pages].to(torch.float64)
        x = x if c["token_major"] else x.permute(0, 2, 1, 3)
        if c["fp8"]:
            x = x * s[name + "s"][pages].double().permute(0, 2, 1).unsqueeze(-1)
        return x.reshape(-1, heads, c["dim"])[:n]

    if c["op"] == "gather":
        lens = _lengths(c["seqs"], c["longest"], c["ragged"])
        return {n: torch.cat([rows(n, b, m) for b, m in enumerate(lens)]) for n in ("k", "v")}
    drafts, ctx = _drafts(c), _lengths(c["batch"], c["longest"], c["ragged"])
    o, lse = s["o"].double(), s["lse"].double()
    for b, (n, t) in enumerate(zip(ctx, drafts)):
        k, v = (rows(name, b, n + t).movedim(0, 1) for name in ("k", "v"))            # [heads, n + t, dim]
        hidden = torch.zeros((t, n + t), dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            hidden[:, n:] = torch.ones((t, t), dtype=torch.bool, device=DEV).triu(1)
        else:
            bits = s["mask"][b, :t].cpu().tolist()
            hidden[:, n:] = torch.tensor([[not (w >> i) & 1 for i in range(t)] for w in bits], device=DEV)
        q = s["q"][b, :t].double().reshape(t, heads, -1, c["dim"]).permute(1, 2, 0, 3)  # [heads, group, t, dim]
        x = q @ k.transpose(-1, -2)[:, None] / math.sqrt(c["dim"])
        x[hidden.expand_as(x)] = -math.inf
        lse[b, :, :t] = torch.logsumexp(x, -1).reshape(-1, t)
        o[b, :t] = (torch.softmax(x, -1) @ v[:, None]).permute(2, 0, 1, 3).reshape(t, -1, c["dim"])
    return {"o": o, "lse": lse}
