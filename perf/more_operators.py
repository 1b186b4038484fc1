"""Measured calls of the prompt and scoring path: rotated appends, chunk attention, windowed layers, log probabilities.

Four operators, each in its plain form (elementary torch operations, 32-bit arithmetic) and through the library's
calls (``own``):

  append    tree_cache_append_rope  new tokens' queries and keys rotated, keys and values written to a paged cache
  chunk     tree_chunk_attn_fwd     attention of the appended chunk over the paged cache, with or without a window
  window    tree_attn_fwd_window    tree attention of a layer with a sliding window and sinks
  logprobs  tree_token_logprobs     log probabilities of given tokens, entropy, the most likely alternatives

A window of W lets position p see the W positions p-W+1 .. p, and the first S ("sinks") besides; W = 0 is no window.
"""
import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------------------- cases

ODD = "0,1,17,130,255,511,700,1001,1300,1537,2000,2222,2500,2999,3333,3700,4001,4096,4444,4800,5003,5500,5901,6144,6500,7000,7123,7400,7777,8000,8100,8191"
PROMPTS = "1024,2047,3111,4096,5000,6143,7001,8192,9215,10240,11111,12288,13001,14336,15359,16384"


def listed():
    return [
        # ordinary decoding: one token for each of 32 sequences of odd lengths, one of them new
        dict(name="append one token", op="append", lens="1*32", prefix=ODD, Hq=32, Hkv=8, D=128, bs=64, q8=False,
             rotary=128, interleaved=False, theta=500000.0, scaling="none", factor=1.0, orig=0),
        # the prompts of a serving batch, straight out of the fused projection
        dict(name="append prompts 1-16K", op="append", lens=PROMPTS, prefix="0*16", Hq=32, Hkv=8, D=128, bs=16, q8=False,
             rotary=128, interleaved=False, theta=500000.0, scaling="bands", factor=8.0, orig=8192),
        # short chunks into the 8-bit cache, adjacent pairs, a quarter of the head
        dict(name="append chunks, 8 bits", op="append", lens="64,1,17,0,33,64,5,48,1,1,64,29,7,64,50,2",
             prefix="1000,77,4096,16383,0,512,2047,9,129,8000,640,31,6001,15,333,12345", Hq=64, Hkv=8, D=128, bs=16,
             q8=True, rotary=32, interleaved=True, theta=10000.0, scaling="ntk", factor=16.0, orig=0),
        # decoding: the newest token of each of the 32 sequences over its cache: bound by reading it
        dict(name="chunk one token", op="chunk", lens="1*32", prefix=ODD, Hq=32, Hkv=8, D=128, bs=64, window=0, sinks=0),
        # a batch that mixes a prompt's next chunk, two short ones and decoding
        dict(name="chunk mixed", op="chunk", lens="1024,1,1,37,1,200,1,1", prefix="2048,8191,4000,0,777,6001,7800,5",
             Hq=32, Hkv=8, D=128, bs=16, window=0, sinks=0),
        # the last 4K tokens of a 16K prompt: bound by the products
        dict(name="chunk 4K of 16K", op="chunk", lens="4096", prefix="12288", Hq=32, Hkv=8, D=128, bs=16, window=0, sinks=0),
        # decoding far into 32K contexts of a windowed layer
        dict(name="chunk one token, window", op="chunk", lens="1*32", prefix="32767*16,20000*16", Hq=32, Hkv=8, D=128,
             bs=64, window=4096, sinks=4),
        # prompt chunks of a windowed layer with heads of 64
        dict(name="chunk 2K, window", op="chunk", lens="2048,1999", prefix="14336,9001", Hq=64, Hkv=8, D=64, bs=16,
             window=4096, sinks=4),
        # the five-node demo tree on 16 tokens with a window of 8: the smallest call
        dict(name="window demo tree", op="window", prefix="16", N=5, Hq=2, Hkv=2, D=64, bs=16, depth=2, window=8, sinks=2),
        # batched serving: 16 sequences, 26-node trees, 1K to 16K tokens, a window of 1K
        dict(name="window batch 16, 1-16K", op="window", prefix=PROMPTS, N=26, Hq=32, Hkv=8, D=128, bs=16, depth=5,
             window=1024, sinks=4),
        # the accepted paths of 16 verified trees, picked out of the trees' logits
        dict(name="logprobs accepted paths", op="logprobs", rows=96, of=416, V=128256, top=8, half=False, temperature=1.0),
        # every token of a 2K prompt
        dict(name="logprobs prompt 2K", op="logprobs", rows=2048, of=2048, V=128256, top=20, half=False, temperature=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "chunk", "window", "logprobs"])
    if op == "logprobs":
        V = rng.choice([1000, 32000, 50257, 128256, _log(rng, 2, 200000)])
        rows = _log(rng, 1, max(1, min(4096, 250_000_000 // V)))
        return dict(op=op, rows=rows, of=rows + rng.choice([0, rng.randint(0, 200)]), V=V, top=min(V, rng.choice([0, 1, 5, 20, 32])),
                    half=rng.random() < 0.5, temperature=rng.choice([1.0, 1.0, 0.7]))
    D = rng.choice([64, 128, 128])
    G = rng.choice([1, 2, 4, 8, 16])
    bs = rng.choice([16, 16, 32, 48, 64, 128, 144])
    window = rng.choice([0, 0, _log(rng, 1, 8192)])
    sinks = rng.choice([0, 4, rng.randint(1, 300)]) if window else 0
    Hkv = rng.choice([1, 2, 8])
    if op == "append":
        q8 = rng.random() < 0.4
        B = _log(rng, 1, 32)
        lens = [0 if rng.random() < 0.1 else _log(rng, 1, 200 if q8 else 16384) for _ in range(B)]
        while sum(lens) * Hkv * (G + 2) > 149000 * 48 or (q8 and sum(lens) > 2048):
            lens = [n // 2 for n in lens]
        lens[0] = max(1, lens[0])
        scaling = rng.choice(["none", "linear", "ntk", "bands"])
        return dict(op=op, lens=",".join(map(str, lens)), prefix=",".join(str(rng.choice([0, _log(rng, 1, 20000)])) for _ in lens),
                    Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs, q8=q8, rotary=rng.choice([D, D, D // 2, 32, 20, 10]),
                    interleaved=rng.random() < 0.5, theta=rng.choice([10000.0, 500000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]), orig=rng.choice([4096, 8192]))
    B = _log(rng, 1, 48)
    top = _log(rng, 64, 65536)
    prefix = [0 if rng.random() < 0.05 else _log(rng, max(1, top // 16), top) for _ in range(B)]
    if op == "window":
        N = rng.choice([1, _log(rng, 1, 256), rng.randint(1, 256)])
        window = window or _log(rng, 1, 8192)
        case = dict(op=op, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs, depth=min(N - 1, rng.randint(0, 12)), window=window, sinks=sinks)
        lens = [N] * B
    else:
        most = rng.choice([1, 1, _log(rng, 1, 4096)])
        lens = [0 if rng.random() < 0.05 else rng.choice([1, _log(rng, 1, most), most]) for _ in range(B)]
        lens[0] = max(1, lens[0])
        case = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs, window=window, sinks=sinks)
    while (_span(prefix, lens, case) * max(lens) * len(lens) * Hkv * G > 4096 * 32 * 16384
           or (sum(prefix) + sum(lens)) * Hkv > 32 * 32768 * 8):
        if max(prefix) > max(lens):
            prefix = [p // 2 for p in prefix]
        elif op == "chunk" and max(lens) > 64:
            lens = [n // 2 for n in lens]
            lens[0] = max(1, lens[0])
        else:
            prefix, lens = prefix[:-1], lens[:-1]
    case["prefix"] = ",".join(map(str, prefix))
    if op == "chunk":
        case["lens"] = ",".join(map(str, lens))
    return case


def _lens(text):
    out = []
    for part in text.split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * (int(times) if times else 1)
    return out


def _far(prefix, case):
    """The first key past the sinks that the first new token may see."""
    return max(case["sinks"], prefix - case["window"] + 1) if case["window"] else 0


def _span(prefixes, lens, case):
    """Keys of the cache, the sinks first, that a sequence's new tokens see at most."""
    new = 0 if case["op"] == "window" else 1
    return case["sinks"] + max(max(0, p + new * n - _far(p, case)) for p, n in zip(prefixes, lens))


# ------------------------------------------------------------------------------------------------------------ inputs

def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _trees(case, B, seed):
    """Random trees of N nodes and the given depth, level by level: parents [B, N] and depths [B, N]."""
    N, top = case["N"], min(case["depth"], case["N"] - 1)
    r = np.random.default_rng([seed, 7])
    lv = np.zeros((B, N), np.int64)
    if N > 1:
        top = max(top, 1)
        lv[:, 1:1 + top] = np.arange(1, top + 1)
        lv[:, 1 + top:] = r.integers(1, top + 1, (B, N - 1 - top))
        lv.sort(axis=1)
    parent = np.full((B, N), -1, np.int32)
    for b in range(B):
        first = np.searchsorted(lv[b], np.arange(top + 2))
        for i in range(1, N):
            parent[b, i] = r.integers(first[lv[b, i] - 1], first[lv[b, i]])
    return parent, lv.astype(np.int32)


def _masks(parent):
    """The ancestor bit masks that tree_build_ancestry gives: [B, N, ceil(N/64)] words."""
    B, N = parent.shape
    words = np.zeros((B, N, (N + 63) // 64), np.uint64)
    for i in range(N):
        if i:
            words[:, i] = words[np.arange(B), parent[:, i]]
        words[:, i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
    return torch.from_numpy(words.view(np.int64)).cuda()


def _paging(lens, bs, seed):
    """A block table for sequences of the given lengths, its blocks in random order; unused entries hold -1."""
    need = [-(-n // bs) for n in lens]
    order = np.random.default_rng([seed, 11]).permutation(max(1, sum(need)))
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), max(1, sum(need))


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "logprobs":
        R, of, V = case["rows"], case["of"], case["V"]
        r = np.random.default_rng([seed, 3])
        x = torch.randn((of, V), generator=g, device="cuda", dtype=torch.float32).mul_(2.5)
        if V > 64:  # some of the vocabulary is masked in every eighth row
            x[::8, V // 3:V // 3 + V // 64] = -math.inf
        s["logits"] = x.to(torch.bfloat16) if case["half"] else x
        s["rows"] = None if of == R else _i32(np.sort(r.choice(of, R, replace=False)))
        s["tokens"] = _i32(r.integers(0, V, R))
        s["logprob"], s["entropy"] = torch.zeros(R, device="cuda"), torch.zeros(R, device="cuda")
        k = case["top"]
        s["top_ids"] = torch.zeros((R, k), dtype=torch.int32, device="cuda") if k else None
        s["top_logprobs"] = torch.zeros((R, k), device="cuda") if k else None
        return s
    D, Hq, Hkv, bs = case["D"], case["Hq"], case["Hkv"], case["bs"]
    prefix = _lens(case["prefix"])
    B = len(prefix)
    lens = _lens(case["lens"]) if "lens" in case else [case["N"]] * B
    T = sum(lens)
    s["status"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["prefix_len"], s["prefix_len_host"] = _i32(prefix), np.array(prefix, np.int32)
    total = prefix if case["op"] == "window" else [p + n for p, n in zip(prefix, lens)]
    s["table"], blocks = _paging(total, bs, seed)
    pool = (blocks, Hkv, bs, D)
    if case["op"] == "append":
        x = _normal(g, (T, Hq + 2 * Hkv, D))  # the projection's output: [q heads | k heads | v heads] of every token
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["q_out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["cu_len"] = _i32(np.concatenate(([0], np.cumsum(lens))))
        dtype = F8 if case["q8"] else torch.bfloat16
        s["k_cache"], s["v_cache"] = torch.zeros(pool, device="cuda").to(dtype), torch.zeros(pool, device="cuda").to(dtype)
        s["scales"] = torch.ones((blocks, Hkv, bs, 2), dtype=torch.uint8, device="cuda") if case["q8"] else None
        return s
    # a hundredth of the keys are eight times the others
    hot = torch.where(torch.rand((blocks, Hkv, bs, 1), generator=g, device="cuda") < 0.01, 8.0, 1.0).to(torch.bfloat16)
    s["k_cache"], s["v_cache"] = _normal(g, pool) * hot, _normal(g, pool)
    if case["op"] == "window":
        N = case["N"]
        s["q"] = _normal(g, (B, N, Hq, D))
        s["k_tree"], s["v_tree"] = _normal(g, (B, N, Hkv, D)), _normal(g, (B, N, Hkv, D))
        parent, depth = _trees(case, B, seed)
        s["mask"], s["depth"] = _masks(parent), torch.from_numpy(depth).cuda()
        s["pos"] = s["prefix_len"][:, None] + s["depth"]
    else:
        s["q"] = _normal(g, (T, Hq, D))
        s["cu_len_host"] = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        s["kv_len_host"] = np.array(total, np.int32)
        s["cu_len"], s["kv_len"] = _i32(s["cu_len_host"]), _i32(total)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(s["q"].shape[:-1], dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------- plain forms

def _frequencies(case):
    """Radians a position for each of the rotary/2 pairs, in 64 bits."""
    R, theta, s = case["rotary"], case["theta"], case["factor"]
    if case["scaling"] == "ntk" and R > 2:
        theta = theta * s ** (R / (R - 2))
    f = theta ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "bands":
        keep = ((case["orig"] * f / (2 * math.pi) - 1.0) / 3.0).clamp(0, 1)  # between 1 and 4 turns in the original context
        f = keep * f + (1 - keep) * f / s
    return f


def _power(biased):
    """2^(biased - 127) in fp32, for biased in [1, 254], without rounding."""
    return (biased.int() << 23).view(torch.float32)


def _quantise(x):
    """Rows of fp32 values (the last axis) to e4m3 codes and scale bytes: value = code * 2^(byte - 127), the power the
    smallest that keeps the row's largest magnitude within 448."""
    mant, exp = torch.frexp(x.abs().amax(dim=-1))  # mant in [0.5, 1)
    byte = torch.where(mant > 0, exp - 9 + (mant > 0.875) + 127, 1).clamp(1, 247)
    return (x * _power(254 - byte)[..., None]).clamp(-448, 448).to(F8), byte.to(torch.uint8)


def _append_out(s):
    out = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_len": s["new_len"]}
    return out if s["scales"] is None else {**out, "scales": s["scales"]}


def _append_plain(s):
    case, R, bs = s["case"], s["case"]["rotary"], s["case"]["bs"]
    n = torch.arange(s["k"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu_len"][1:].contiguous(), n.int(), right=True)
    pos = s["prefix_len"][seq] + n - s["cu_len"][seq]
    s["new_len"].copy_(s["prefix_len"] + s["cu_len"].diff())
    angle = pos.double()[:, None, None] * _frequencies(case)  # 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()

    def turn(x):
        x = x.float()
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
        y, z = a * cos - b * sin, b * cos + a * sin
        y = torch.stack((y, z), dim=-1).flatten(-2) if case["interleaved"] else torch.cat((y, z), dim=-1)
        return torch.cat((y, x[..., R:]), dim=-1).to(torch.bfloat16)

    s["q_out"].copy_(turn(s["q"]))
    blk, row = s["table"][seq, pos // bs].long(), pos % bs
    k = turn(s["k"])
    if s["scales"] is None:
        s["k_cache"][blk, :, row] = k
        s["v_cache"][blk, :, row] = s["v"]
    else:
        for x, cache, which in ((k, "k_cache", 0), (s["v"], "v_cache", 1)):
            codes, byte = _quantise(x.float())
            s[cache].view(torch.uint8)[blk, :, row] = codes.view(torch.uint8)
            s["scales"][blk, :, row, which] = byte
    return _append_out(s)


def _keys(s, lens):
    """The cache rows that a sequence's new tokens may see, the sinks first: fp32 [B, S, Hkv, D] of keys and of values,
    and their positions [B, 1, S]; those past the sequence (or twice there) are at 2^30."""
    case, bs = s["case"], s["case"]["bs"]
    prefix = s["prefix_len_host"].tolist()
    total = s["prefix_len"] if case["op"] == "window" else s["kv_len"]
    j = torch.arange(max(1, _span(prefix, lens, case)), device="cuda")[None]
    first = _i32([_far(p, case) for p in prefix])[:, None]
    t = torch.where(j < case["sinks"], j, first + j - case["sinks"])
    seen = (t < total[:, None]) & ((j >= case["sinks"]) | (j < first))
    blk = s["table"].gather(1, (t // bs).clamp(max=s["table"].shape[1] - 1).long()).clamp(min=0).long()
    row = (t % bs).long()
    t = torch.where(seen, t, 1 << 30)
    k, v = (s[c][blk, :, row].float() for c in ("k_cache", "v_cache"))
    return k, torch.where(seen[..., None, None], v, 0.0), t[:, None]


def _near(case, pos, t):
    """Whether the key at t is within reach of the row at pos."""
    return t <= pos if not case["window"] else (t <= pos) & ((t > pos - case["window"]) | (t < case["sinks"]))


def _heads(x, G):
    """Rows [B, N, Hq, D] as [B, Hkv, N * G, D], and scores' row masks to match come from repeat_interleave."""
    B, N, Hq, D = x.shape
    return x.view(B, N, Hq // G, G, D).transpose(1, 2).reshape(B, Hq // G, N * G, D)


def _back(x, N, G):
    B, Hkv, _, D = x.shape
    return x.view(B, Hkv, N, G, D).transpose(1, 2).reshape(B, N, Hkv * G, D)


def _attend(q, groups):
    """One softmax over groups of (keys [B, Hkv, D, S], values [B, Hkv, S, D], mask [B, 1, rows, S]); q [B, Hkv, rows, D]."""
    scores = [(q @ k).masked_fill_(~m, -math.inf) for k, _, m in groups]
    top = torch.stack([x.amax(dim=-1) for x in scores]).amax(dim=0)[..., None].clamp(min=-3e38)
    scores = [x.sub_(top).exp_() for x in scores]
    total = sum(x.sum(dim=-1, keepdim=True) for x in scores)
    out = sum(x @ v for x, (_, v, _) in zip(scores, groups)) / total
    return out, top + total.log()


def _chunk_plain(s):
    case, D = s["case"], s["case"]["D"]
    G = case["Hq"] // case["Hkv"]
    lens = s["cu_len_host"][1:] - s["cu_len_host"][:-1]
    N = int(lens.max())
    i = torch.arange(N, device="cuda")[None]
    own_row = i < s["cu_len"].diff()[:, None]  # sequences padded to the longest
    at = torch.where(own_row, s["cu_len"][:-1, None] + i, 0).long()
    pos = torch.where(own_row, s["prefix_len"][:, None] + i, 1 << 29)
    k, v, t = _keys(s, lens.tolist())
    mask = _near(case, pos[..., None], t) if case["window"] else t <= pos[..., None]
    mask = (mask | ~own_row[..., None]).repeat_interleave(G, dim=1)[:, None]
    o, lse = _attend(_heads(s["q"][at].float() * D ** -0.5, G), [(k.permute(0, 2, 3, 1), v.transpose(1, 2), mask)])
    s["out"].copy_(_back(o, N, G)[own_row])
    s["lse"].copy_(_back(lse, N, G)[own_row].squeeze(-1))
    return {"out": s["out"], "lse": s["lse"]}


def _window_plain(s):
    case, N, D = s["case"], s["case"]["N"], s["case"]["D"]
    G = case["Hq"] // case["Hkv"]
    k, v, t = _keys(s, [N] * s["q"].shape[0])
    far = _near(case, s["pos"][..., None], t)
    j = torch.arange(N, device="cuda")
    seen = ((s["mask"][:, :, j // 64] >> (j % 64)) & 1) != 0
    seen &= _near(case, s["pos"][..., None], s["pos"][:, None])
    far, seen = (m.repeat_interleave(G, dim=1)[:, None] for m in (far, seen))
    o, lse = _attend(_heads(s["q"].float() * D ** -0.5, G), [
        (k.permute(0, 2, 3, 1), v.transpose(1, 2), far),
        (s["k_tree"].float().permute(0, 2, 3, 1), s["v_tree"].float().transpose(1, 2), seen)])
    s["out"].copy_(_back(o, N, G))
    s["lse"].copy_(_back(lse, N, G).squeeze(-1))
    return {"out": s["out"], "lse": s["lse"]}


def _logprobs_out(s):
    out = {"logprob": s["logprob"], "entropy": s["entropy"]}
    return out if s["top_ids"] is None else {**out, "top_ids": s["top_ids"], "top_logprobs": s["top_logprobs"]}


def _logprobs_plain(s):
    case = s["case"]
    raw = s["logits"] if s["rows"] is None else s["logits"][s["rows"].long()]
    x = raw.float() / case["temperature"]
    top = x.amax(dim=-1, keepdim=True)
    y = x - top
    e = y.exp()
    total = e.sum(dim=-1, keepdim=True)
    log_total = total.log()
    s["logprob"].copy_((y.gather(1, s["tokens"].long()[:, None]) - log_total)[:, 0])
    s["entropy"].copy_((log_total - (e * y.clamp(min=-3e38)).sum(dim=-1, keepdim=True) / total)[:, 0])
    if case["top"]:
        # by value, then by the lower index: the float's bits in order, above the index counted down
        bits = raw.float().add(0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits)
        key = (order << 32) + ((1 << 31) - 1 - torch.arange(case["V"], device="cuda"))
        ids = (1 << 31) - 1 - (key.topk(case["top"], dim=-1).values & 0xFFFFFFFF)
        val = y.gather(1, ids) - log_total
        s["top_ids"].copy_(torch.where(val > -math.inf, ids, -1))  # a masked token is no alternative
        s["top_logprobs"].copy_(val)
    return _logprobs_out(s)


# ---------------------------------------------------------------------------------------------- the library's calls

def _run_own(s):
    import tree_attention_speculative_gb300 as ts
    case = s["case"]
    if case["op"] == "append":
        if "rope" not in s:  # kept by the program, as its model's configuration is
            s["rope"] = ts.RopeConfig(theta=case["theta"], rotary_dim=case["rotary"], interleaved=case["interleaved"],
                                      scaling=case["scaling"], factor=case["factor"], low_rot=1.0, high_rot=4.0,
                                      orig_len=case["orig"])
        ts.tree_cache_append_rope(s["q"], s["k"], s["v"], s["cu_len"], s["prefix_len"], s["q_out"], s["k_cache"],
                                  s["v_cache"], s["table"], s["new_len"], s["rope"], status=s["status"], kv_scale=s["scales"])
        return _append_out(s)
    if case["op"] == "logprobs":
        ts.tree_token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], top_ids=s["top_ids"],
                               top_logprobs=s["top_logprobs"], rows=s["rows"], temperature=case["temperature"])
        return _logprobs_out(s)
    if case["op"] == "chunk":
        p = ts.chunk_params(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu_len"], s["kv_len"], s["cu_len_host"],
                            s["kv_len_host"], s["out"], s["lse"], s["status"], window=case["window"], sinks=case["sinks"])
        if "workspace" not in s:  # zero-filled once, kept by the program
            s["workspace"] = torch.zeros(ts.tree_chunk_attn_workspace_size(p), dtype=torch.uint8, device="cuda")
        ts.tree_chunk_attn_fwd(p, s["workspace"])
    else:
        p = ts.attn_params(s["q"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], s["prefix_len_host"],
                           s["k_tree"], s["v_tree"], s["mask"], s["pos"], s["out"], s["lse"], s["status"])
        if "workspace" not in s:
            size = ts.tree_attn_window_workspace_size(p, case["window"], case["sinks"])
            s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        ts.tree_attn_fwd_window(p, case["window"], case["sinks"], s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append_plain, "chunk": _chunk_plain, "window": _window_plain, "logprobs": _logprobs_plain}[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------- what a pass cannot do without

def _pairs(prefix, n, case):
    """(row, key) pairs of a chunk of n tokens after `prefix`, and how many keys any of its rows sees."""
    pos = np.arange(prefix, prefix + n, dtype=np.int64)
    if not case["window"]:
        return int((pos + 1).sum()), prefix + n if n else 0
    W, S = case["window"], case["sinks"]
    near = np.minimum(pos + 1, W)
    far = np.minimum(S, np.maximum(0, pos + 1 - W))
    lo = max(0, prefix - W + 1)
    return int((near + far).sum()), prefix + n - lo + min(S, lo) if n else 0


def work(case):
    if case["op"] == "logprobs":
        R, V = case["rows"], case["V"]
        return {"bytes": R * V * (2 if case["half"] else 4) + R * (12 + 8 * case["top"]), "flops": 5 * R * V}
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    prefix = _lens(case["prefix"])
    B = len(prefix)
    if case["op"] == "append":
        T = sum(_lens(case["lens"]))
        row = 2 * (D + 1) if case["q8"] else 4 * D
        return {"bytes": T * (2 * (Hq + 2 * Hkv) * D + 2 * Hq * D + Hkv * row) + 24 * B, "flops": 3 * T * (Hq + Hkv) * case["rotary"]}
    if case["op"] == "window":
        N, W = case["N"], case["window"]
        keys = [min(p, W - 1) + min(case["sinks"], max(0, p - W + 1)) for p in prefix]
        tree = B * N * (2 * Hkv * D * 2 + 8 * ((N + 63) // 64))
        return {"bytes": sum(keys) * Hkv * 4 * D + tree + B * N * Hq * (4 * D + 4), "flops": 4 * D * Hq * N * (sum(keys) + B)}
    lens = _lens(case["lens"])
    pairs, keys = (sum(x) for x in zip(*(_pairs(p, n, case) for p, n in zip(prefix, lens))))
    return {"bytes": keys * Hkv * 4 * D + 4 * sum(-(-k // case["bs"]) for k in prefix) + sum(lens) * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------------------ the definitions in 64 bits

def _exact_logprobs(s):
    case = s["case"]
    R, k = case["rows"], case["top"]
    pick = np.arange(R) if s["rows"] is None else s["rows"].cpu().numpy()
    logp, ent = (torch.empty(R, dtype=torch.float64, device="cuda") for _ in range(2))
    ids = torch.full((R, k), -1, dtype=torch.int32, device="cuda")
    alt = torch.full((R, k), -math.inf, dtype=torch.float64, device="cuda")
    for lo in range(0, R, 64):
        x = s["logits"][torch.from_numpy(pick[lo:lo + 64]).long().cuda()].double() / case["temperature"]
        n = torch.log_softmax(x, dim=-1)
        logp[lo:lo + 64] = n.gather(1, s["tokens"][lo:lo + 64].long()[:, None])[:, 0]
        ent[lo:lo + 64] = -torch.special.xlogy(n.exp(), n.exp()).sum(dim=-1)
        if k:
            val, at = torch.sort(n, dim=-1, descending=True, stable=True)
            val, at = val[:, :k], at[:, :k].int()
            ids[lo:lo + 64], alt[lo:lo + 64] = torch.where(val > -math.inf, at, -1), val
    out = {"logprob": logp, "entropy": ent}
    return {**out, "top_ids": ids, "top_logprobs": alt} if k else out


def _two_to(e):
    """2^e as doubles, exactly, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest_e4m3(x):
    """The e4m3 value next to x (a double within +-448), ties to the even code."""
    _, e = torch.frexp(x)
    step = (e - 4).clamp(min=-9)  # the codes around x are 2^step apart
    return torch.round(x * _two_to(-step)) * _two_to(step)  # torch.round: halves to even


def _exact_append(s):
    case, R, bs = s["case"], s["case"]["rotary"], s["case"]["bs"]
    theta = case["theta"] * (case["factor"] ** (R / (R - 2)) if case["scaling"] == "ntk" and R > 2 else 1.0)
    freq = []
    for i in range(R // 2):
        f = math.exp(-2 * i / R * math.log(theta))
        if case["scaling"] == "linear":
            f /= case["factor"]
        elif case["scaling"] == "bands":
            turns = case["orig"] * f / (2 * math.pi)
            f = f if turns >= 4 else f / case["factor"] if turns <= 1 else f * ((turns - 1) / 3 + (4 - turns) / 3 / case["factor"])
        freq.append(f)
    freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
    cu, prefix = s["cu_len"].tolist(), s["prefix_len"].tolist()
    q = s["q_out"].double()
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    scales = None if s["scales"] is None else s["scales"].clone()
    for b, p in enumerate(prefix):
        n = cu[b + 1] - cu[b]
        if not n:
            continue
        t = torch.arange(p, p + n, device="cuda")
        angle = t.double()[:, None, None] * freq
        unit = torch.polar(torch.ones_like(angle), angle)

        def turn(x):
            x = x.double().clone()
            pairs = x[..., :R].unflatten(-1, (R // 2, 2)) if case["interleaved"] else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
            x[..., :R] = (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)
            return x

        q[cu[b]:cu[b + 1]] = turn(s["q"][cu[b]:cu[b + 1]])
        blk = s["table"][b].long()[t // bs]
        for x, cache, which in ((turn(s["k"][cu[b]:cu[b + 1]]), k_cache, 0), (s["v"][cu[b]:cu[b + 1]].double(), v_cache, 1)):
            if scales is not None:
                x = x.to(torch.bfloat16).double()  # rotated keys are bf16 before they are stored
                largest = x.abs().amax(dim=-1, keepdim=True).clamp(min=1e-38)
                e = torch.ceil(torch.log2(largest / 448))
                e = torch.where(448 * _two_to(e - 1) >= largest, e - 1, e)  # whatever log2 rounds to
                e = torch.where(448 * _two_to(e) < largest, e + 1, e).clamp(min=-126)
                x = _nearest_e4m3(x * _two_to(-e))
                scales[blk, :, t % bs, which] = (e.squeeze(-1) + 127).to(torch.uint8)
            cache[blk, :, t % bs] = x
    out = {"q": q, "k_cache": k_cache, "v_cache": v_cache, "new_len": s["prefix_len"] + s["cu_len"].diff()}
    return out if scales is None else {**out, "scales": scales}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    if case["op"] == "append":
        return _exact_append(s)
    D, Hkv, bs, W, S = case["D"], case["Hkv"], case["bs"], case["window"], case["sinks"]
    G = case["Hq"] // Hkv
    out, lse = s["out"].double(), s["lse"].double()
    for b, p in enumerate(s["prefix_len_host"].tolist()):
        if case["op"] == "window":
            q, o, l, kv = s["q"][b], out[b], lse[b], p
            pos = s["pos"][b].long()
            bits = s["mask"][b].cpu().numpy().view(np.uint8).reshape(case["N"], -1)
            related = torch.from_numpy(np.unpackbits(bits, axis=1, bitorder="little")[:, :case["N"]].astype(bool)).cuda()
        else:
            lo, hi = s["cu_len_host"][b], s["cu_len_host"][b + 1]
            q, o, l, kv = s["q"][lo:hi], out[lo:hi], lse[lo:hi], int(s["kv_len_host"][b])
            pos = torch.arange(p, kv, device="cuda")
        if not len(pos):
            continue
        at = torch.arange(kv, device="cuda")
        allowed = at[None] <= pos[:, None]
        if case["op"] == "window":
            at = torch.cat((at, pos))
            allowed = torch.cat((allowed, related), dim=1)
        if W:
            allowed = allowed & ((pos[:, None] - at[None] < W) | (at[None] < S))
        blocks = s["table"][b, :-(-kv // bs)].long()
        for g in range(Hkv):
            keys, values = (s[c][blocks, g].reshape(-1, D)[:kv].double() for c in ("k_cache", "v_cache"))
            if case["op"] == "window":
                keys = torch.cat((keys, s["k_tree"][b, :, g].double()))
                values = torch.cat((values, s["v_tree"][b, :, g].double()))
            for h in range(g * G, (g + 1) * G):
                logits = (q[:, h].double() @ keys.T) / math.sqrt(D)
                logits = torch.where(allowed, logits, torch.full_like(logits, -math.inf))
                l[:, h] = torch.logsumexp(logits, dim=1)
                o[:, h] = torch.exp(logits - l[:, h, None]) @ values
    return {"out": out, "lse": lse}
