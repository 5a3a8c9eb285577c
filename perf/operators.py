"""Measured cases of the cache-writing and 4-bit operators.

Three operators, each through the package's public calls where `own` is true
and in elementary torch operations where it is not:

  rotate_append  per-head norm and rotary position of q and k, and the append
                 of k and v to a paged bf16 or fp32 cache (norm_rope_append)
  append4        the append to a cache held in 4 bits (norm_rope_append)
  attend4        attention over a cache held in 4 bits (attend_varlen)

4-bit pools are uint8 (num_blocks, kv_heads, 9 * head_dim): 8 * head_dim bytes
of e2m1 codes (two a byte) of a page's 16 tokens, then head_dim bytes of
scales, one for 16 consecutive columns of a token, as unsigned e5m3 floats.
A K page lists its tokens in order.  A V page is stored the other way round:
byte `hi` of column d of token pair t holds tokens 2t + 8hi (low nibble) and
2t + 8hi + 1, so that a pair of tokens is one byte.
"""
import math
import random

import torch

own = False

PAGE = 16


# ---------------------------------------------------------------- cases

def listed():
    rope = {"op": "rotate_append", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot_dim": 128, "interleaved": False,
            "norm": False, "scaling": "none", "segments": 1, "q_len": 1, "ragged": False, "kv_len": 8192, "far": False}
    app = {"op": "append4", "kv_heads": 8, "head_dim": 128, "segments": 1, "q_len": 1, "ragged": False, "kv_len": 8192}
    att = {"op": "attend4", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "segments": 1, "q_len": 1, "ragged": False, "kv_len": 300,
           "causal": False, "window": 0, "ring": False}
    return [
        # one token of one sequence: the decode step of a single chat, all latency
        {"name": "rope one token", **rope},
        # a decode step of a large batch whose model normalises q and k for each head, frequencies scaled for a long context
        {"name": "rope norm batch", **rope, "norm": True, "scaling": "yarn", "segments": 256, "kv_len": 512},
        # prompts of uneven length going in: interleaved pairs on half the head, positions far beyond the trained context
        {"name": "rope prompts ragged", **rope, "norm": True, "scaling": "linear", "rot_dim": 64, "interleaved": True, "segments": 5, "q_len": 4099,
         "ragged": True, "kv_len": 5003, "far": True},
        # the small fp32 configuration, a few draft tokens for each sequence
        {"name": "rope fp32 drafts", **rope, "dtype": "f32", "q_heads": 8, "kv_heads": 2, "head_dim": 64, "rot_dim": 64, "segments": 3, "q_len": 7,
         "ragged": True, "kv_len": 509},
        # one token of one sequence into a 4-bit cache
        {"name": "append4 one token", **app},
        # uneven prompts into a 4-bit cache
        {"name": "append4 prompts ragged", **app, "segments": 16, "q_len": 2039, "ragged": True, "kv_len": 4096},
        # a young sequence: latency of the smallest attention
        {"name": "attend4 short", **att},
        # one sequence at the largest fixed bucket
        {"name": "attend4 bucket 8192", **att, "kv_len": 8192},
        # a decode step of uneven sequences: bandwidth
        {"name": "attend4 batch varlen", **att, "segments": 32, "ragged": True, "kv_len": 16384},
        # draft tokens checked in one step: wide row groups
        {"name": "attend4 drafts causal", **att, "q_heads": 64, "segments": 16, "q_len": 16, "ragged": True, "kv_len": 8192, "causal": True},
        # long contexts with wide heads
        {"name": "attend4 long", **att, "kv_heads": 4, "head_dim": 256, "segments": 4, "kv_len": 131072},
        # the same contexts behind a sliding window in ring storage
        {"name": "attend4 long window", **att, "kv_heads": 4, "head_dim": 256, "segments": 4, "kv_len": 131072, "causal": True, "window": 4096, "ring": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate_append", "rotate_append", "append4", "attend4", "attend4", "attend4"])
    hq, hkv = rng.choice([(32, 8), (64, 8), (8, 2), (16, 16), (32, 4), (12, 3), (7, 1), (40, 8)])
    if op == "rotate_append":
        d = rng.choice([64, 80, 128, 128, 256])
        s = _log(rng, 1, 256)
        n = _log(rng, 1, max(1, 16384 // s))
        kv = n + _log(rng, 1, max(1, min(4096, (1 << 27) // (s * hkv * d) - n))) - 1
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]), "q_heads": hq, "kv_heads": hkv, "head_dim": d,
                "rot_dim": rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]), "interleaved": rng.random() < 0.4,
                "norm": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "yarn"]), "segments": s, "q_len": n,
                "ragged": rng.random() < 0.7, "kv_len": kv, "far": rng.random() < 0.3}
    d = rng.choice([64, 128, 128, 256])
    if op == "append4":
        s = _log(rng, 1, 256)
        n = _log(rng, 1, max(1, 16384 // s))
        kv = n + _log(rng, 1, max(1, min(4096, (1 << 28) // (s * hkv * d) - n))) - 1
        return {"op": op, "kv_heads": hkv, "head_dim": d, "segments": s, "q_len": n, "ragged": rng.random() < 0.7, "kv_len": kv}
    s = _log(rng, 1, 64)
    n = 1 if rng.random() < 0.6 else _log(rng, 2, 32)
    most = min(131072, (1 << 28) // (s * hkv * d), 4_000_000_000 // (s * n * hq * d))
    kv = max(n, _log(rng, 16, max(16, most)))
    window = 0 if rng.random() < 0.6 else _log(rng, 16, max(16, kv))
    return {"op": op, "q_heads": hq, "kv_heads": hkv, "head_dim": d, "segments": s, "q_len": n, "ragged": rng.random() < 0.7, "kv_len": kv,
            "causal": rng.random() < 0.5, "window": window, "ring": window > 0 and rng.random() < 0.5}


def _lengths(case):
    """(q_len, kv_end) of each segment: a matter of the case, not of the seed."""
    n, kv, s = case["q_len"], case["kv_len"], case["segments"]
    if not case["ragged"]:
        return [(n, kv)] * s
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    q = [r.randint(1, n) for _ in range(s - 1)] + [n]
    return [(a, r.randint(a, kv)) for a in q[:-1]] + [(n, kv)]


def _ring(case):
    return -(-(case["window"] + case["q_len"] - 1) // PAGE) * PAGE if case.get("ring") else 0


def _key_range(case, n, kv):
    """The keys [lo, kv) that a segment of n rows reads."""
    w = case.get("window", 0)
    if not w:
        return 0
    return max(0, (kv - n if case["causal"] else kv - 1) - w + 1)


def work(case):
    d, hkv, lens = case["head_dim"], case["kv_heads"], _lengths(case)
    rows = sum(n for n, _ in lens)
    if case["op"] == "rotate_append":
        e = 2 if case["dtype"] == "bf16" else 4
        heads = case["q_heads"] + 2 * hkv
        flops = rows * (case["q_heads"] + hkv) * (3 * case["rot_dim"] + (4 * d if case["norm"] else 0))
        return {"bytes": 2 * rows * heads * d * e + 16 * len(lens) + 8 * rows, "flops": flops}
    if case["op"] == "append4":  # rows in, rows as stored out, codes and scales out
        return {"bytes": rows * 2 * hkv * d * (2 + 2 + 9 / 16) + 16 * len(lens), "flops": rows * 2 * hkv * d * 4}
    hq = case["q_heads"]
    keys = sum(kv - _key_range(case, n, kv) for n, kv in lens)
    pairs = 0
    for n, kv in lens:
        for i in range(n):
            hi = kv - n + i + 1 if case["causal"] else kv
            pairs += hi - (max(0, hi - case["window"]) if case["window"] else 0)
    return {"bytes": keys * hkv * 2 * d * 9 / 16 + rows * hq * (4 * d + 4) + keys / 4, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------- inputs

def _inv_freq(case):
    """Angles a position, in 64 bits, and the factor on cos and sin: plain, stretched, or stretched by parts (YaRN)."""
    r = case["rot_dim"]
    f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if case["scaling"] == "linear":
        return f / 8.0, 1.0
    if case["scaling"] == "yarn":
        factor, trained = 16.0, 8192.0
        turns = trained * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)  # 1: turns often enough in the trained context to stay
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens = _lengths(case)
    rows, ring = sum(n for n, _ in lens), _ring(case)
    used = [ring // PAGE if ring else -(-kv // PAGE) for _, kv in lens]
    blocks, width = sum(used) + 3, max(used) + 1
    ids = torch.randperm(blocks, generator=g, device=dev)[:sum(used)].to(torch.int32).cpu()
    table, info, at, q0 = torch.full((len(lens), width), -1, dtype=torch.int32), [], 0, 0
    for i, (n, kv) in enumerate(lens):
        table[i, :used[i]] = ids[at:at + used[i]]
        info.append([q0, n, i, kv])
        at, q0 = at + used[i], q0 + n
    d, hkv = case["head_dim"], case["kv_heads"]
    s = {"op": case["op"], "case": case, "table": table.to(dev), "seq_info": torch.tensor(info, dtype=torch.int32, device=dev), "ring": ring,
         "max_q": case["q_len"], "heads": (case.get("q_heads", 0), hkv, d), "rows": rows}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    spread = torch.exp(0.5 * normal(hkv, 1, d))  # some columns of K are larger than others
    if case["op"] == "rotate_append":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["k"], s["v"] = [normal(blocks, PAGE, hkv, d).to(dt) for _ in range(2)]
        s["q"] = (1.5 * normal(rows, case["q_heads"], d)).to(dt)
        s["k_new"], s["v_new"] = (normal(rows, hkv, d) * spread.view(hkv, d)).to(dt), (0.5 * normal(rows, hkv, d)).to(dt)
        s["q_out"] = torch.empty_like(s["q"])
        f, s["mscale"] = _inv_freq(case)
        s["inv_freq"], s["eps"] = f.to(dev), 1e-6
        s["q_weight"], s["k_weight"] = [(1 + 0.2 * normal(d)).to(dt) if case["norm"] else None for _ in range(2)]
        s["positions"] = torch.randint(0, 1 << 20, (rows,), generator=g, device=dev, dtype=torch.int32) if case["far"] else None
    else:
        s["k"], s["v"] = torch.empty(blocks, hkv, 9 * d, dtype=torch.uint8, device=dev), torch.empty(blocks, hkv, 9 * d, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 26) // (hkv * PAGE * d))
        for b in range(0, blocks, step):
            n = min(step, blocks - b)
            s["k"][b:b + n] = _pack_k(*_quantise(normal(n, hkv, PAGE, d) * spread))
            s["v"][b:b + n] = _pack_v(*_quantise(0.5 * normal(n, hkv, PAGE, d)))
        if case["op"] == "append4":
            s["k_new"] = (normal(rows, hkv, d) * spread.view(hkv, d)).bfloat16()
            s["v_new"] = (0.5 * normal(rows, hkv, d)).bfloat16()
            s["k_out"], s["v_out"] = torch.empty_like(s["k_new"]), torch.empty_like(s["v_new"])
            s["pages"] = (case["q_len"] + PAGE - 2) // PAGE + 1  # pages that a segment's new rows reach, at most
        else:
            s["q"] = (2.0 / spread.view(hkv, 1, d) * normal(rows, hkv, case["q_heads"] // hkv, d)).reshape(rows, -1, d).bfloat16()
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(rows, case["q_heads"], dtype=torch.float32, device=dev)
            s["scale"] = d ** -0.5
            longest = max(kv - _key_range(case, n, kv) for n, kv in lens)
            s["pages"] = (longest + PAGE - 2) // PAGE + 1
    if own:
        import paged_kv_decode_13_gb300 as pkv
        s["pkv"] = pkv
        s["cache"] = pkv.PagedKVCache([s["k"]], [s["v"]], s["table"], ring_rows=ring)
        s["err"] = pkv.new_err_flags(dev)
        if case["op"] == "rotate_append":
            s["rope"] = pkv.Rope(s["inv_freq"], interleaved=case["interleaved"], mscale=s["mscale"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                 eps=s["eps"])
    return s


# ---------------------------------------------------------------- the 4-bit format

def _quantise(x):
    """Codes (uint8, 0..15) and scale bytes of fp32 rows [..., d]: s = e5m3(max|x| / 6), code = e2m1(x / s), both to nearest even."""
    x = x.unflatten(-1, (-1, 16))
    a = x.abs().amax(-1) / 6.0
    bits = a.view(torch.int32)
    normal = (((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) << 20).view(torch.float32)
    s = torch.where(a < 2.0 ** -14, torch.round(a * 2.0 ** 17) * 2.0 ** -17, normal).clamp(max=10240.0)
    r = torch.where(s[..., None] > 0, x.abs() / s[..., None], torch.zeros_like(x))
    mag = ((r > 0.25).to(torch.uint8) + (r >= 0.75).to(torch.uint8) + (r > 1.25).to(torch.uint8) + (r >= 1.75).to(torch.uint8)
           + (r > 2.5).to(torch.uint8) + (r >= 3.5).to(torch.uint8) + (r > 5.0).to(torch.uint8))
    codes = mag | (torch.signbit(x).to(torch.uint8) << 3)
    return codes.flatten(-2), (s.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)


def _values(codes, scales):
    """fp32 values of codes [..., d] and their scale bytes [..., d / 16]."""
    c = (codes & 7).float()  # 0 0.5 1 1.5 2 3 4 6: the step doubles at 2 and at 4
    v = 0.5 * (c + (c - 4).clamp(min=0)) + (c - 6).clamp(min=0)
    v = torch.where(codes >= 8, -v, v)
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _pack_k(codes, scales):
    """[..., 16, d] codes and [..., 16, d / 16] scales to K blocks [..., 9 d]."""
    return torch.cat([(codes[..., 0::2] | (codes[..., 1::2] << 4)).flatten(-2), scales.flatten(-2)], -1)


def _unpack_k(block):
    d = block.shape[-1] // 9
    b = block[..., :8 * d].unflatten(-1, (16, d // 2))
    return torch.stack([b & 15, b >> 4], -1).flatten(-2), block[..., 8 * d:].unflatten(-1, (16, d // 16))


def _pack_v(codes, scales):
    """The same for V blocks: token = 8 hi + 2 t + nibble, column = (d / 8) g + 8 p + i, byte (p, g, t, i, hi)."""
    d = codes.shape[-1]
    c = codes.unflatten(-1, (8, d // 64, 8)).unflatten(-4, (2, 4, 2))  # hi t nibble g p i
    b = c[..., 0, :, :, :] | (c[..., 1, :, :, :] << 4)  # hi t g p i
    b = b.movedim((-2, -3, -4, -1, -5), (-5, -4, -3, -2, -1)).flatten(-5)
    s = scales.unflatten(-2, (2, 4, 2)).movedim((-1, -3, -4, -2), (-4, -3, -2, -1)).flatten(-4)  # group t hi nibble
    return torch.cat([b, s], -1)


def _unpack_v(block):
    d = block.shape[-1] // 9
    b = block[..., :8 * d].unflatten(-1, (d // 64, 8, 4, 8, 2)).movedim((-5, -4, -3, -2, -1), (-2, -3, -4, -1, -5))  # hi t g p i
    c = torch.stack([b & 15, b >> 4], -4).flatten(-6, -4).flatten(-3)
    s = block[..., 8 * d:].unflatten(-1, (d // 16, 4, 2, 2)).movedim((-4, -3, -2, -1), (-1, -3, -4, -2)).flatten(-4, -2)
    return c, s


# ---------------------------------------------------------------- the plain forms

def _row_places(s):
    """(segment, position) of every row."""
    info = s["seq_info"].long()
    row = torch.arange(s["rows"], device=info.device)
    seg = torch.searchsorted(info[:, 0].contiguous(), row, right=True) - 1
    return seg, info[seg, 3] - info[seg, 1] + row - info[seg, 0]


def _rotate(x, weight, s, pos):
    """Per-head norm (where there is a weight) and rotary position of rows [rows, heads, d], in fp32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    angle = pos.double()[:, None] * s["inv_freq"]
    c, t = [(s["mscale"] * f(angle)).float()[:, None, :] for f in (torch.cos, torch.sin)]
    r = 2 * s["inv_freq"].numel()
    if s["case"]["interleaved"]:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        return torch.cat([torch.stack([u * c - v * t, v * c + u * t], -1).flatten(-2), x[..., r:]], -1)
    u, v = x[..., :r // 2], x[..., r // 2:r]
    return torch.cat([u * c - v * t, v * c + u * t, x[..., r:]], -1)


def _rotate_append(s):
    seg, place = _row_places(s)
    pos = place if s["positions"] is None else s["positions"]
    q = _rotate(s["q"], s["q_weight"], s, pos).to(s["q"].dtype)
    k = _rotate(s["k_new"], s["k_weight"], s, pos).to(s["k"].dtype)
    block = s["table"].long()[seg, place // PAGE]
    s["k"][block, place % PAGE] = k
    s["v"][block, place % PAGE] = s["v_new"]
    return q, s["k"], s["v"]


def _append4(s):
    info = s["seq_info"].long()
    start, end = info[:, 3] - info[:, 1], info[:, 3]
    page = torch.minimum(start[:, None] // PAGE + torch.arange(s["pages"], device=info.device), (end[:, None] - 1) // PAGE)  # the last one repeats
    block = s["table"].long().gather(1, page)
    token = page[..., None] * PAGE + torch.arange(PAGE, device=info.device)
    new = (token >= start[:, None, None]) & (token < end[:, None, None])
    row = (info[:, 0, None, None] + token - start[:, None, None]).clamp(0, s["rows"] - 1)
    out = []
    for name, pack, unpack in (("k", _pack_k, _unpack_k), ("v", _pack_v, _unpack_v)):
        codes, scales = _quantise(s[name + "_new"].float())
        out.append(_values(codes, scales).bfloat16())
        old_codes, old_scales = unpack(s[name][block])
        m = new[:, :, None, :, None]
        s[name][block] = pack(torch.where(m, codes[row].transpose(2, 3), old_codes), torch.where(m, scales[row].transpose(2, 3), old_scales))
    return out[0], out[1], s["k"], s["v"]


def _attend4(s):
    hq, hkv, d = s["heads"]
    causal, window = s["case"]["causal"], s["case"]["window"]
    dev = s["q"].device
    info = s["seq_info"].long()
    q0, n, col, end = info.unbind(1)
    start = end - n
    i = torch.arange(s["max_q"], device=dev)
    pos = start[:, None] + i  # of the rows
    hi = pos + 1 if causal else end[:, None].expand_as(pos)
    lo = (hi - window).clamp(min=0) if window else torch.zeros_like(hi)
    page = lo[:, :1] // PAGE + torch.arange(s["pages"], device=dev)
    slot = page % (s["ring"] // PAGE) if s["ring"] else page
    block = s["table"].long()[col].gather(1, slot.clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k, v = [_values(*u(s[p][block])).transpose(1, 2).flatten(2, 3) for p, u in (("k", _unpack_k), ("v", _unpack_v))]  # [s, heads, keys, d]
    key = (page[..., None] * PAGE + torch.arange(PAGE, device=dev)).flatten(1)
    q = s["q"][(q0[:, None] + i).clamp(max=s["rows"] - 1)].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    seen = (key[:, None, :] >= lo[..., None]) & (key[:, None, :] < hi[..., None])
    x = x.masked_fill(~seen.repeat_interleave(hq // hkv, 1)[:, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total
    lse = m + torch.log(total)
    row = torch.where(i < n[:, None], q0[:, None] + i, s["rows"])  # rows of no segment go to a spare one
    back = lambda t: t.unflatten(2, (-1, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # noqa: E731
    whole, sums = torch.zeros(s["rows"] + 1, hq, d, device=dev), torch.zeros(s["rows"] + 1, hq, 1, device=dev)
    whole[row], sums[row] = back(out), back(lse)
    return whole[:-1].bfloat16(), sums[:-1, :, 0]


def run(state):
    s = state
    if not own:
        return {"rotate_append": _rotate_append, "append4": _append4, "attend4": _attend4}[s["op"]](s)
    pkv = s["pkv"]
    if s["op"] == "rotate_append":
        pkv.norm_rope_append(s["cache"], 0, s["rope"], s["q"], s["k_new"], s["v_new"], s["seq_info"], s["q_out"], s["err"], positions=s["positions"])
        return s["q_out"], s["k"], s["v"]
    if s["op"] == "append4":
        pkv.norm_rope_append(s["cache"], 0, None, None, s["k_new"], s["v_new"], s["seq_info"], None, s["err"], k_out=s["k_out"], v_out=s["v_out"])
        return s["k_out"], s["v_out"], s["k"], s["v"]
    c = s["case"]
    pkv.attend_varlen(s["cache"], 0, s["q"], s["seq_info"], s["out"], s["err"], s["max_q"], c["kv_len"], s["scale"], c["causal"], c["window"], lse=s["lse"])
    return s["out"], s["lse"]


# ---------------------------------------------------------------- the definition, in 64 bits

def _exact_block(block, d, values):
    """The 64-bit values of pages [pages, heads, 9 d] as [heads, pages * 16, d], by the place of each code and scale."""
    key, col = torch.meshgrid(torch.arange(PAGE), torch.arange(d), indexing="ij")
    if values:
        g, i, t, hi, nib = col // (d // 8), col % (d // 8), key % 8 // 2, key // 8, key % 2
        at, scale = i // 8 * 512 + (g * 4 + t) * 16 + i % 8 * 2 + hi, 8 * d + (col // 16 * 4 + t) * 4 + hi * 2 + nib
    else:
        at, nib, scale = key * (d // 2) + col // 2, col % 2, 8 * d + key * (d // 16) + col // 16
    at, nib, scale = at.to(block.device), nib.to(block.device), scale.to(block.device)
    code, b = (block[..., at] >> (4 * nib).to(torch.uint8)) & 15, block[..., scale].long()
    e, m = (code.long() & 7) >> 1, code.long() & 1
    mag = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2((e - 1).double()))
    s = torch.where(b < 8, b.double() * 2.0 ** -17, (8 + b % 8).double() * torch.exp2((b // 8 - 18).double()))
    return torch.where(code >= 8, -mag * s, mag * s).permute(1, 0, 2, 3).reshape(block.shape[1], -1, d)


def _exact_stored(x):
    """What a row is stored as: the nearest scale of all of them, then the nearest value of the eight."""
    x = x.double().unflatten(-1, (-1, 16))
    dev = x.device
    scales = torch.tensor([(b * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18)) for b in range(227)], dtype=torch.float64, device=dev)
    a = x.abs().amax(-1) / 6

    def nearest(v, grid):
        i = torch.searchsorted(grid, v).clamp(1, len(grid) - 1)
        below, above = v - grid[i - 1], grid[i] - v
        return torch.where((below < above) | ((below == above) & ((i - 1) % 2 == 0)), i - 1, i)

    s = scales[nearest(a, scales)]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev)
    mag = grid[nearest((x.abs() / s[..., None]).nan_to_num(0.0, posinf=0.0), grid)]
    return torch.copysign(mag * s[..., None], x).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    lens = _lengths(case)
    hq, hkv, d = s["heads"]
    if case["op"] == "append4":
        return _exact_stored(s["k_new"]), _exact_stored(s["v_new"]), None, None
    table = s["table"].long()
    if case["op"] == "rotate_append":
        pools, q = [s["k"].double(), s["v"].double()], []
        at = 0
        for j, (n, kv) in enumerate(lens):
            place = torch.arange(kv - n, kv, device=table.device)
            pos = (place if s["positions"] is None else s["positions"][at:at + n].long()).double()
            turn = torch.polar(torch.full((n, case["rot_dim"] // 2), s["mscale"], dtype=torch.float64, device=table.device), pos[:, None] * s["inv_freq"])
            got = []
            for x, w in ((s["q"], s["q_weight"]), (s["k_new"], s["k_weight"])):
                x = x[at:at + n].double()
                if w is not None:
                    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.double()
                y, r = x.clone(), case["rot_dim"]
                a, b = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
                z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
                y[..., a], y[..., b] = z.real, z.imag
                got.append(y)
            q.append(got[0])
            pools[0][table[j, place // PAGE], place % PAGE] = got[1]
            pools[1][table[j, place // PAGE], place % PAGE] = s["v_new"][at:at + n].double()
            at += n
        return torch.cat(q), pools[0], pools[1]
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device=table.device)
    lse = torch.zeros(s["rows"], hq, dtype=torch.float64, device=table.device)
    at = 0
    for j, (n, kv) in enumerate(lens):
        first = _key_range(case, n, kv) // PAGE
        pages = torch.arange(first, -(-kv // PAGE), device=table.device)
        ids = table[j, pages % (s["ring"] // PAGE) if s["ring"] else pages]
        k, v = _exact_block(s["k"][ids], d, False), _exact_block(s["v"][ids], d, True)
        key = first * PAGE + torch.arange(k.shape[1], device=table.device)
        hi = torch.arange(kv - n + 1, kv + 1, device=table.device) if case["causal"] else torch.full((n,), kv, device=table.device)
        lo = (hi - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(hi)
        hide = (key[None, :] < lo[:, None]) | (key[None, :] >= hi[:, None])
        for h in range(hq):
            x = s["scale"] * (s["q"][at:at + n, h].double() @ k[h // (hq // hkv)].T)
            x = torch.where(hide, float("-inf"), x)
            lse[at:at + n, h] = torch.logsumexp(x, -1)
            out[at:at + n, h] = torch.exp(x - lse[at:at + n, h, None]).nan_to_num(0.0) @ torch.where((key < kv)[:, None], v[h // (hq // hkv)], 0.0)
        at += n
    return out, lse
