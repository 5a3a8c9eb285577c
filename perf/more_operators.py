"""Measured cases of positions with several axes, the 8-bit cache and attention over whole prompts.

Four operators, each through the package's public calls where `own` is true
and in elementary torch operations where it is not:

  rotate_axes  per-head norm and rotary position of q and k with an axis for
               each pair of columns, with the append to a bf16 or fp32 cache
               (norm_rope_append) or for rows that go to none (norm_rope)
  append8      the append to a cache held in 8 bits, and the new rows as it
               holds them (norm_rope_append)
  attend8      attention over a cache held in 8 bits (attend_varlen)
  prompt       attention of packed prompts over their own rows (attend_prompt)

8-bit pools are float8_e4m3fn (num_blocks, kv_heads, 16 * head_dim + 16): a
page's 16 tokens as e4m3 codes, then 16 bytes of which the first is the
exponent e + 127 of the scale 2^e of that page and kv head (0: no scale, all
values zero), the third and fourth mark tokens that hold a NaN, and the others
are not used.  The scale is the smallest power of two by which every value of
the page fits e4m3's 448; tokens that are in the page already keep it from
getting smaller, and are brought to the larger one.  The 16-byte chunk c of
token t is in place c ^ (((t & 6) ^ (t & 1) << 2) % (head_dim / 16)) of its row.
"""
import math
import random

import torch

own = False

PAGE = 16


# ---------------------------------------------------------------- cases

def listed():
    rope = {"op": "rotate_axes", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot_dim": 128, "axes": 3, "dealt": False,
            "interleaved": False, "norm": False, "cached": True, "segments": 1, "q_len": 1, "ragged": False, "kv_len": 8192}
    app = {"op": "append8", "kv_heads": 8, "head_dim": 128, "segments": 1, "q_len": 1, "ragged": False, "kv_len": 8192}
    att = {"op": "attend8", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "segments": 1, "q_len": 1, "ragged": False, "kv_len": 300,
           "causal": False, "window": 0, "ring": False}
    pro = {"op": "prompt", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "segments": 1, "q_len": 8192, "ragged": False, "causal": True,
           "window": 0, "fused": False}
    return [
        # one token of a chat that has had images: three positions a row, all latency
        {"name": "axes one token", **rope},
        # prompts of text and images going in, time, height and width dealt to the pairs in turn
        {"name": "axes prompts ragged", **rope, "norm": True, "dealt": True, "segments": 5, "q_len": 4099, "ragged": True, "kv_len": 5003},
        # an image encoder's patches: height and width, heads of 80 columns, no cache
        {"name": "axes patches", **rope, "q_heads": 16, "kv_heads": 16, "head_dim": 80, "rot_dim": 80, "axes": 2, "cached": False, "segments": 3,
         "q_len": 2500, "ragged": True, "kv_len": 2500},
        # a decode step of a large batch into an 8-bit cache: pages that are partly full
        {"name": "append8 batch", **app, "segments": 256, "ragged": True, "kv_len": 512},
        # uneven prompts into an 8-bit cache
        {"name": "append8 prompts ragged", **app, "segments": 16, "q_len": 2039, "ragged": True, "kv_len": 4096},
        # a young sequence: latency of the smallest attention
        {"name": "attend8 short", **att},
        # a decode step of uneven sequences: bandwidth
        {"name": "attend8 batch varlen", **att, "segments": 32, "ragged": True, "kv_len": 16384},
        # draft tokens checked in one step: wide row groups
        {"name": "attend8 drafts causal", **att, "q_heads": 64, "segments": 16, "q_len": 16, "ragged": True, "kv_len": 8192, "causal": True},
        # long contexts with wide heads
        {"name": "attend8 long", **att, "kv_heads": 4, "head_dim": 256, "segments": 4, "kv_len": 131072},
        # short questions packed together, q, k and v as slices of one projection's output
        {"name": "prompt short ragged", **pro, "segments": 16, "q_len": 301, "ragged": True, "fused": True},
        # one prompt that fills the largest fixed bucket
        {"name": "prompt 8192", **pro},
        # uneven prompts behind a sliding window, wide heads
        {"name": "prompt window wide", **pro, "kv_heads": 4, "head_dim": 256, "segments": 4, "q_len": 4096, "ragged": True, "window": 1024},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate_axes", "append8", "attend8", "attend8", "prompt", "prompt"])
    hq, hkv = rng.choice([(32, 8), (64, 8), (8, 2), (16, 16), (32, 4), (12, 3), (7, 1), (40, 8)])
    if op == "rotate_axes":
        d = rng.choice([64, 80, 128, 128, 256])
        s = _log(rng, 1, 256)
        n = _log(rng, 1, max(1, 16384 // s))
        kv = n + _log(rng, 1, max(1, min(4096, (1 << 27) // (s * hkv * d) - n))) - 1
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(4, d // 2)])
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]), "q_heads": hq, "kv_heads": hkv, "head_dim": d, "rot_dim": rot,
                "axes": rng.choice([2, 3, 3, 4]), "dealt": rng.random() < 0.5, "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.5,
                "cached": rng.random() < 0.7, "segments": s, "q_len": n, "ragged": rng.random() < 0.7, "kv_len": kv}
    d = rng.choice([64, 128, 128, 256])
    if op == "append8":
        s = _log(rng, 1, 256)
        n = _log(rng, 1, max(1, 16384 // s))
        kv = n + _log(rng, 1, max(1, min(4096, (1 << 28) // (s * hkv * d) - n))) - 1
        return {"op": op, "kv_heads": hkv, "head_dim": d, "segments": s, "q_len": n, "ragged": rng.random() < 0.7, "kv_len": kv}
    if op == "prompt":
        d = rng.choice([64, 80, 128, 128, 256])
        s = _log(rng, 1, 64)
        n = _log(rng, 1, min(8192, int(math.sqrt((1 << 31) * min(1.0, 128 / d) / (s * hq)))))
        return {"op": op, "q_heads": hq, "kv_heads": hkv, "head_dim": d, "segments": s, "q_len": n, "ragged": rng.random() < 0.7,
                "causal": rng.random() < 0.8, "window": 0 if rng.random() < 0.6 else _log(rng, 1, 4096), "fused": rng.random() < 0.5}
    s = _log(rng, 1, 64)
    n = 1 if rng.random() < 0.6 else _log(rng, 2, 32)
    most = min(131072, (1 << 28) // (s * hkv * d), 4_000_000_000 // (s * n * hq * d))
    kv = max(n, _log(rng, 16, max(16, most)))
    window = 0 if rng.random() < 0.6 else _log(rng, 16, max(16, kv))
    return {"op": op, "q_heads": hq, "kv_heads": hkv, "head_dim": d, "segments": s, "q_len": n, "ragged": rng.random() < 0.7, "kv_len": kv,
            "causal": rng.random() < 0.5, "window": window, "ring": window > 0 and rng.random() < 0.5}


def _lengths(case):
    """(q_len, kv_end) of each segment: a matter of the case, not of the seed."""
    n, s = case["q_len"], case["segments"]
    kv = case.get("kv_len", n)
    if not case["ragged"]:
        return [(n, kv)] * s
    r = random.Random(str(sorted((k, v) for k, v in case.items() if k != "name")))
    q = [r.randint(1, n) for _ in range(s - 1)] + [n]
    if case["op"] == "prompt":
        return [(a, a) for a in q]
    return [(a, r.randint(a, kv)) for a in q[:-1]] + [(n, kv)]


def _ring(case):
    return -(-(case["window"] + case["q_len"] - 1) // PAGE) * PAGE if case.get("ring") else 0


def _key_range(case, n, kv):
    """The first key that a segment of n rows reads."""
    w = case.get("window", 0)
    if not w:
        return 0
    return max(0, (kv - n if case["causal"] else kv - 1) - w + 1)


def _pairs(case, n, kv):
    """(row, key) pairs that a segment's rows see."""
    w, total = case["window"], 0
    for i in range(n):
        hi = kv - n + i + 1 if case["causal"] else kv
        total += hi - (max(0, hi - w) if w else 0)
    return total


def work(case):
    d, hkv, lens = case["head_dim"], case["kv_heads"], _lengths(case)
    rows = sum(n for n, _ in lens)
    if case["op"] == "rotate_axes":
        e = 2 if case["dtype"] == "bf16" else 4
        heads = case["q_heads"] + (2 if case["cached"] else 1) * hkv
        flops = rows * (case["q_heads"] + hkv) * (3 * case["rot_dim"] + (4 * d if case["norm"] else 0))
        return {"bytes": 2 * rows * heads * d * e + 4 * rows * case["axes"] + 16 * len(lens), "flops": flops}
    if case["op"] == "append8":  # rows in, rows as held out, codes out
        return {"bytes": rows * 2 * hkv * d * (2 + 2 + 1) + 16 * len(lens), "flops": rows * 2 * hkv * d * 4}
    hq = case["q_heads"]
    pairs = sum(_pairs(case, n, kv) for n, kv in lens)
    if case["op"] == "prompt":
        return {"bytes": rows * (4 * hq * d + 4 * hkv * d + 4 * hq), "flops": 4 * pairs * hq * d}
    keys = sum(kv - _key_range(case, n, kv) for n, kv in lens)
    return {"bytes": keys * hkv * 2 * (d + 1) + rows * hq * (4 * d + 4) + keys / 4, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------- inputs

def _sections(case):
    """Pairs of each axis: even shares, the first axis with what is left over."""
    n, a = case["rot_dim"] // 2, case["axes"]
    return [n - (a - 1) * (n // a)] + [n // a] * (a - 1)


def _axis_of_pair(case):
    """The axis that turns each pair: axis after axis, or dealt in turn to those that have pairs left."""
    left, out = _sections(case), []
    if not case["dealt"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens = _lengths(case)
    rows, ring = sum(n for n, _ in lens), _ring(case)
    d, hkv = case["head_dim"], case["kv_heads"]
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    pooled = op in ("append8", "attend8") or (op == "rotate_axes" and case["cached"])
    used = [(ring // PAGE if ring else -(-kv // PAGE)) if pooled else 0 for _, kv in lens]
    blocks, width = sum(used) + 3, max(used) + 1
    ids = torch.randperm(blocks, generator=g, device=dev)[:sum(used)].to(torch.int32).cpu()
    table, info, at, q0 = torch.full((len(lens), width), -1, dtype=torch.int32), [], 0, 0
    for i, (n, kv) in enumerate(lens):
        table[i, :used[i]] = ids[at:at + used[i]]
        info.append([q0, n, i, kv])
        at, q0 = at + used[i], q0 + n
    s = {"op": op, "case": case, "table": table.to(dev), "seq_info": torch.tensor(info, dtype=torch.int32, device=dev), "ring": ring,
         "max_q": case["q_len"], "heads": (case.get("q_heads", 0), hkv, d), "rows": rows}
    spread = torch.exp(0.5 * normal(hkv, 1, d))  # some columns of K are larger than others
    if op == "rotate_axes":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["q"] = (1.5 * normal(rows, case["q_heads"], d)).to(dt)
        s["k_new"] = (normal(rows, hkv, d) * spread.view(hkv, d)).to(dt)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k_new"])
        if pooled:
            s["k"], s["v"] = [normal(blocks, PAGE, hkv, d).to(dt) for _ in range(2)]
            s["v_new"] = (0.5 * normal(rows, hkv, d)).to(dt)
        pairs = case["rot_dim"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=dev) / pairs)
        s["axis"] = torch.tensor(_axis_of_pair(case), device=dev)
        s["eps"] = 1e-6
        s["q_weight"], s["k_weight"] = [(1 + 0.2 * normal(d)).to(dt) if case["norm"] else None for _ in range(2)]
        # time goes on with the rows, the others run over a picture of up to 64 places a side
        first = torch.randint(0, 1 << 15, (1,), generator=g, device=dev, dtype=torch.int32)
        places = torch.randint(0, 64, (rows, case["axes"] - 1), generator=g, device=dev, dtype=torch.int32)
        time = first + torch.arange(rows, device=dev, dtype=torch.int32)[:, None]
        s["positions"] = torch.cat([time, time // 2 + places], 1).contiguous()
    elif op == "prompt":
        hq = case["q_heads"]
        if case["fused"]:
            qkv = torch.empty(rows, hq + 2 * hkv, d, dtype=torch.bfloat16, device=dev)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=dev)
            s["k"], s["v"] = [torch.empty(rows, hkv, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        s["q"].copy_((2.0 / spread.view(hkv, 1, d) * normal(rows, hkv, hq // hkv, d)).reshape(rows, hq, d))
        s["k"].copy_(normal(rows, hkv, d) * spread.view(hkv, d))
        s["v"].copy_(0.5 * normal(rows, hkv, d))
        s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device=dev)
        s["scale"] = d ** -0.5
    else:
        s["k"], s["v"] = [torch.zeros(blocks, hkv, PAGE * d + 16, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
        step = max(1, (1 << 26) // (hkv * PAGE * d))
        for b in range(0, blocks, step):
            n = min(step, blocks - b)
            for name, x in (("k", normal(n, hkv, PAGE, d) * spread), ("v", 0.5 * normal(n, hkv, PAGE, d))):
                x = (x * torch.exp(0.7 * normal(n, hkv, 1, 1))).bfloat16().float()  # some pages are larger than others
                e = _exponent(x.abs().amax((-2, -1)))
                s[name].view(torch.uint8)[b:b + n] = _pack(_codes(x, e[..., None, None]), e, d)
        if op == "append8":
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
        s["err"] = pkv.new_err_flags(dev)
        if pooled:
            s["cache"] = pkv.PagedKVCache([s["k"]], [s["v"]], s["table"], ring_rows=ring)
        if op == "rotate_axes":
            s["rope"] = pkv.Rope(s["inv_freq"], interleaved=case["interleaved"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                                 axes=pkv.rope_axes(_sections(case), dealt=case["dealt"]))
    return s


# ---------------------------------------------------------------- the 8-bit format

def _exponent(largest):
    """The exponent bytes of blocks whose largest magnitudes are given: the smallest e with largest <= 448 * 2^e, as e + 127; 0 for all zeros."""
    m, e = torch.frexp(largest)  # m in [0.5, 1), 448 = 0.875 * 2^9
    b = (e - 9 + (m > 0.875).to(e.dtype) + 127).clamp(1, 246)
    return torch.where(largest > 0, b, torch.zeros_like(b))


def _scale(b):
    return torch.where(b > 0, torch.exp2((b - 127).float()), torch.zeros((), device=b.device))


def _codes(x, b):
    """e4m3 codes of fp32 values under the exponent bytes b."""
    return (x * torch.exp2((127 - b).float())).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _places(d, device):
    """The byte of (token, column) in a block."""
    t, c = torch.arange(PAGE, device=device)[:, None], torch.arange(d, device=device)
    return t * d + 16 * ((c // 16) ^ (((t & 6) ^ ((t & 1) << 2)) % (d // 16))) + c % 16


def _pack(codes, b, d):
    """[..., 16, d] codes and [...] exponent bytes to blocks [..., 16 d + 16]."""
    out = torch.zeros(*b.shape, PAGE * d + 16, dtype=torch.uint8, device=b.device)
    out[..., _places(d, b.device)] = codes
    out[..., PAGE * d] = b.to(torch.uint8)
    return out


def _unpack(block):
    """Blocks to codes [..., 16, d] and exponent bytes [...]."""
    d = (block.shape[-1] - 16) // PAGE
    return block[..., _places(d, block.device)], block[..., PAGE * d].int()


# ---------------------------------------------------------------- the plain forms

def _rotate(x, weight, s, pos):
    """Per-head norm (where there is a weight) and rotary position of rows [rows, heads, d], in fp32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    angle = pos[:, s["axis"]].double() * s["inv_freq"]
    c, t = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    r = 2 * s["inv_freq"].numel()
    if s["case"]["interleaved"]:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        return torch.cat([torch.stack([u * c - v * t, v * c + u * t], -1).flatten(-2), x[..., r:]], -1)
    u, v = x[..., :r // 2], x[..., r // 2:r]
    return torch.cat([u * c - v * t, v * c + u * t, x[..., r:]], -1)


def _rotate_axes(s):
    q = _rotate(s["q"], s["q_weight"], s, s["positions"]).to(s["q"].dtype)
    k = _rotate(s["k_new"], s["k_weight"], s, s["positions"]).to(s["q"].dtype)
    if not s["case"]["cached"]:
        return q, k
    info = s["seq_info"].long()
    row = torch.arange(s["rows"], device=info.device)
    seg = torch.searchsorted(info[:, 0].contiguous(), row, right=True) - 1
    place = info[seg, 3] - info[seg, 1] + row - info[seg, 0]
    block = s["table"].long()[seg, place // PAGE]
    s["k"][block, place % PAGE] = k
    s["v"][block, place % PAGE] = s["v_new"]
    return q, s["k"], s["v"]


def _append8(s):
    info = s["seq_info"].long()
    _, hkv, d = s["heads"]
    start, end = info[:, 3] - info[:, 1], info[:, 3]
    page = torch.minimum(start[:, None] // PAGE + torch.arange(s["pages"], device=info.device), (end[:, None] - 1) // PAGE)  # the last one repeats
    block = s["table"].long().gather(1, page)
    token = page[..., None] * PAGE + torch.arange(PAGE, device=info.device)
    new = (token >= start[:, None, None]) & (token < end[:, None, None])
    kept = token < start[:, None, None]
    row = (info[:, 0, None, None] + token - start[:, None, None]).clamp(0, s["rows"] - 1)
    spare = torch.where(new, row, s["rows"])
    n, k = new[:, :, None, :, None], kept[:, :, None, :, None]
    out = []
    for name in ("k", "v"):
        pool = s[name].view(torch.uint8)
        blk = pool[block]  # [segments, pages, heads, bytes]
        old, e0 = _unpack(blk)
        x = torch.where(n, s[name + "_new"].float()[row].transpose(2, 3), 0.0)
        e = torch.maximum(_exponent(x.abs().amax((-2, -1))), torch.where(kept.any(-1)[..., None], e0, 0))
        have = old.view(torch.float8_e4m3fn).float() * _scale(e0)[..., None, None]
        codes = torch.where(n, _codes(x, e[..., None, None]), torch.where(k, _codes(have, e[..., None, None]), old))
        held = torch.zeros(s["rows"] + 1, hkv, d, dtype=torch.bfloat16, device=info.device)
        held[spare] = (codes.view(torch.float8_e4m3fn).float() * _scale(e)[..., None, None]).bfloat16().transpose(2, 3)
        out.append(held[:-1])
        pool[block] = _pack(codes, e, d)
    return out[0], out[1], s["k"].view(torch.uint8), s["v"].view(torch.uint8)


def _softmax_rows(x, seen, v):
    """Weighted sums of v by the softmax of the seen scores, and the log of the sum of exponentials; x is used up."""
    x.masked_fill_(~seen, float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x.sub_(m), out=x)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total, m + torch.log(total)


def _bounds(s, start, n, end):
    """Positions of the rows of each segment and their keys [lo, hi)."""
    i = torch.arange(s["max_q"], device=start.device)
    pos = start[:, None] + i
    hi = pos + 1 if s["case"]["causal"] else end[:, None].expand_as(pos)
    w = s["case"]["window"]
    return i, (hi - w).clamp(min=0) if w else torch.zeros_like(hi), hi


def _scatter(s, out, lse, i, q0, n):
    """[segments, kv heads, rows * group, ..] back to packed rows."""
    hq, hkv, d = s["heads"]
    row = torch.where(i < n[:, None], q0[:, None] + i, s["rows"])  # rows of no segment go to a spare one
    back = lambda t: t.unflatten(2, (-1, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # noqa: E731
    whole, sums = torch.zeros(s["rows"] + 1, hq, d, device=q0.device), torch.zeros(s["rows"] + 1, hq, 1, device=q0.device)
    whole[row], sums[row] = back(out), back(lse)
    return whole[:-1].bfloat16(), sums[:-1, :, 0]


def _attend8(s):
    hq, hkv, d = s["heads"]
    dev = s["q"].device
    q0, n, col, end = s["seq_info"].long().unbind(1)
    i, lo, hi = _bounds(s, end - n, n, end)
    page = lo[:, :1] // PAGE + torch.arange(s["pages"], device=dev)
    slot = page % (s["ring"] // PAGE) if s["ring"] else page
    block = s["table"].long()[col].gather(1, slot.clamp(max=s["table"].shape[1] - 1)).clamp(min=0)

    def values(pool):
        codes, e = _unpack(pool.view(torch.uint8)[block])
        return (codes.view(torch.float8_e4m3fn).float() * _scale(e)[..., None, None]).transpose(1, 2).flatten(2, 3)  # [s, heads, keys, d]

    key = (page[..., None] * PAGE + torch.arange(PAGE, device=dev)).flatten(1)
    q = s["q"][(q0[:, None] + i).clamp(max=s["rows"] - 1)].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(q, values(s["k"]).transpose(2, 3)).mul_(s["scale"])
    seen = (key[:, None, :] >= lo[..., None]) & (key[:, None, :] < hi[..., None])
    out, lse = _softmax_rows(x, seen.repeat_interleave(hq // hkv, 1)[:, None], values(s["v"]))
    return _scatter(s, out, lse, i, q0, n)


def _prompt(s):
    hq, hkv, d = s["heads"]
    q0, n, _, end = s["seq_info"].long().unbind(1)
    i, lo, hi = _bounds(s, end - n, n, end)
    row = (q0[:, None] + i).clamp(max=s["rows"] - 1)
    k, v = [s[name][row].float().transpose(1, 2) for name in ("k", "v")]  # [segments, heads, keys, d]
    q = s["q"][row].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    seen = (i >= lo[..., None]) & (i < torch.minimum(hi, n[:, None])[..., None])
    out, lse = _softmax_rows(x, seen.repeat_interleave(hq // hkv, 1)[:, None], v)
    return _scatter(s, out, lse, i, q0, n)


def run(state):
    s = state
    if not own:
        return {"rotate_axes": _rotate_axes, "append8": _append8, "attend8": _attend8, "prompt": _prompt}[s["op"]](s)
    pkv, c = s["pkv"], s["case"]
    if s["op"] == "rotate_axes" and c["cached"]:
        pkv.norm_rope_append(s["cache"], 0, s["rope"], s["q"], s["k_new"], s["v_new"], s["seq_info"], s["q_out"], s["err"], positions=s["positions"])
        return s["q_out"], s["k"], s["v"]
    if s["op"] == "rotate_axes":
        pkv.norm_rope(s["rope"], s["q"], s["k_new"], s["positions"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    if s["op"] == "append8":
        pkv.norm_rope_append(s["cache"], 0, None, None, s["k_new"], s["v_new"], s["seq_info"], None, s["err"], k_out=s["k_out"], v_out=s["v_out"])
        return s["k_out"], s["v_out"], s["k"].view(torch.uint8), s["v"].view(torch.uint8)
    if s["op"] == "attend8":
        pkv.attend_varlen(s["cache"], 0, s["q"], s["seq_info"], s["out"], s["err"], s["max_q"], c["kv_len"], s["scale"], c["causal"], c["window"], lse=s["lse"])
    else:
        pkv.attend_prompt(s["q"], s["k"], s["v"], s["seq_info"], s["out"], s["err"], s["max_q"], s["scale"], c["causal"], c["window"], lse=s["lse"])
    return s["out"], s["lse"]


# ---------------------------------------------------------------- the definition, in 64 bits

def _e4m3(codes):
    """The 64-bit numbers of e4m3 codes, by their fields."""
    c = codes.long()
    e, m = (c >> 3) & 15, c & 7
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    return torch.where(c >= 128, -mag, mag)


def _exact_pages(blocks, d):
    """[pages, heads, 16 d + 16] as 64-bit values [heads, pages * 16, d], token after token."""
    out = []
    for t in range(PAGE):
        f = ((t & 6) ^ (4 if t & 1 else 0)) % (d // 16)
        row = blocks[..., t * d:(t + 1) * d].unflatten(-1, (-1, 16))
        out.append(row[..., [c ^ f for c in range(d // 16)], :].flatten(-2))
    e = blocks[..., PAGE * d].double()
    s = torch.where(e > 0, torch.exp2(e - 127), torch.zeros_like(e))
    return (_e4m3(torch.stack(out, -2)) * s[..., None, None]).transpose(0, 1).flatten(1, 2)


def _exact_held(x, floor):
    """What rows [n, heads, d] of one page are held as: under the smallest power of two by which the largest fits, at least `floor`; nearest codes, ties to even."""
    x = x.double()
    big = x.abs().amax((0, 2))
    s = torch.exp2(torch.round(torch.log2(big.clamp(min=2.0 ** -117) / 448)))
    s = torch.where(big > 448 * s, 2 * s, torch.where(big <= 224 * s, s / 2, s))
    s = torch.maximum(torch.where(big > 0, s, torch.zeros_like(s)), floor)
    grid = _e4m3(torch.arange(127, device=x.device))
    r = torch.where(s[None, :, None] > 0, x.abs() / s[None, :, None], torch.zeros_like(x)).contiguous()
    i = torch.searchsorted(grid, r).clamp(1, 126)
    below, above = r - grid[i - 1], grid[i] - r
    i = torch.where((below < above) | ((below == above) & ((i - 1) % 2 == 0)), i - 1, i)
    return torch.copysign(grid[i] * s[None, :, None], x)


def _exact_attention(q, k, v, scale, lo, hi, key, out, lse):
    """Rows q [n, heads, d] over k and v [kv heads, keys, d], whose positions are `key`, into out and lse."""
    group = q.shape[1] // k.shape[0]
    hide = (key[None, :] < lo[:, None]) | (key[None, :] >= hi[:, None])
    used = (~hide).any(0)[:, None]
    for h in range(q.shape[1]):
        x = scale * (q[:, h].double() @ k[h // group].double().T)
        x.masked_fill_(hide, float("-inf"))
        lse[:, h] = torch.logsumexp(x, -1)
        out[:, h] = torch.exp(x - lse[:, h, None]).nan_to_num(0.0) @ torch.where(used, v[h // group].double(), 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    lens = _lengths(case)
    hq, hkv, d = s["heads"]
    table = s["table"].long()
    dev = table.device
    at = 0
    if case["op"] == "append8":
        got = [torch.zeros(s["rows"], hkv, d, dtype=torch.float64, device=dev) for _ in range(2)]
        if sum(-(-n // PAGE) + 1 for n, _ in lens) > 4000:
            return None
        for j, (n, kv) in enumerate(lens):
            for p in range((kv - n) // PAGE, -(-kv // PAGE)):
                a, b = max(p * PAGE, kv - n), min((p + 1) * PAGE, kv)
                for name, out in (("k", got[0]), ("v", got[1])):
                    e = s[name].view(torch.uint8)[table[j, p], :, PAGE * d].double()
                    floor = torch.where(e > 0, torch.exp2(e - 127), torch.zeros_like(e)) if a > p * PAGE else torch.zeros_like(e)
                    r = slice(at + a - (kv - n), at + b - (kv - n))
                    out[r] = _exact_held(s[name + "_new"][r], floor)
            at += n
        return got[0], got[1], None, None
    if case["op"] == "rotate_axes":
        pos, axis = s["positions"].double(), _axis_of_pair(case)
        angle = torch.stack([pos[:, a] * s["inv_freq"][i] for i, a in enumerate(axis)], 1)
        turn = torch.polar(torch.ones_like(angle), angle)
        got = []
        for x, w in ((s["q"], s["q_weight"]), (s["k_new"], s["k_weight"])):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.double()
            y, r = x.clone(), case["rot_dim"]
            a, b = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(x[..., a], x[..., b]) * turn[:, None]
            y[..., a], y[..., b] = z.real, z.imag
            got.append(y)
        if not case["cached"]:
            return got[0], got[1]
        pools = [s["k"].double(), s["v"].double()]
        for j, (n, kv) in enumerate(lens):
            place = torch.arange(kv - n, kv, device=dev)
            pools[0][table[j, place // PAGE], place % PAGE] = got[1][at:at + n]
            pools[1][table[j, place // PAGE], place % PAGE] = s["v_new"][at:at + n].double()
            at += n
        return got[0], pools[0], pools[1]
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["rows"], hq, dtype=torch.float64, device=dev)
    for j, (n, kv) in enumerate(lens):
        hi = torch.arange(kv - n + 1, kv + 1, device=dev) if case["causal"] else torch.full((n,), kv, device=dev)
        lo = (hi - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(hi)
        r = slice(at, at + n)
        if case["op"] == "prompt":
            k, v = s["k"][r].transpose(0, 1), s["v"][r].transpose(0, 1)
            key = torch.arange(n, device=dev)
        else:
            first = _key_range(case, n, kv) // PAGE
            pages = torch.arange(first, -(-kv // PAGE), device=dev)
            ids = table[j, pages % (s["ring"] // PAGE) if s["ring"] else pages]
            k, v = [_exact_pages(s[name].view(torch.uint8)[ids], d) for name in ("k", "v")]
            key = first * PAGE + torch.arange(k.shape[1], device=dev)
        _exact_attention(s["q"][r], k, v, s["scale"], lo, hi, key, out[r], lse[r])
        at += n
    return out, lse
