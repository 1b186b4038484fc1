"""Measured calls of the 8-bit cache path: rotary positions, quantised cache writes, attention over the 8-bit cache.

Four operators, each in its plain form (elementary torch operations, 32-bit arithmetic) and through the library's
calls (``own``):

  rope     tree_rope               q and k rotated at their positions, read out of a fused projection or dense
  append   tree_cache_append_q8    prompt tokens quantised to e4m3 as they are written to a paged cache
  commit   tree_commit_accepted_q8 a verified path quantised as it is committed
  attn     tree_attn_fwd_q8        tree attention over the quantised paged prefix and the bf16 tree block

A cache row (one token of one KV head, D values) is stored as e4m3 codes and one scale byte s: value = code * 2^(s - 127),
the power of two being the smallest that keeps the row's largest magnitude within 448.
"""
import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the five-node demo tree (2 heads of 64): what a call costs when there is nothing to do
        dict(name="rope demo tree", op="rope", B=1, N=5, Hq=2, Hkv=2, D=64, rotary=64, interleaved=False, fused=False,
             theta=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, orig=0, mscale=1.0, start=16),
        # a 70B-shaped layer, 64 sequences of 64 nodes past 8K tokens, straight out of the fused projection, with
        # frequencies scaled by bands for a longer context
        dict(name="rope batch 64, fused", op="rope", B=64, N=64, Hq=64, Hkv=8, D=128, rotary=128, interleaved=False,
             fused=True, theta=500000.0, scaling="bands", factor=8.0, low=1.0, high=4.0, orig=8192, mscale=1.0, start=8192),
        # four 192-node trees past 128K tokens; adjacent pairs, a quarter of the head, base scaled
        dict(name="rope 128K, partial", op="rope", B=4, N=192, Hq=32, Hkv=8, D=128, rotary=32, interleaved=True,
             fused=False, theta=10000.0, scaling="ntk", factor=16.0, low=1.0, high=4.0, orig=0, mscale=1.0, start=131072),
        # ordinary decoding beside the trees: one token for each of 16 sequences
        dict(name="append one token", op="append", lens="1*16", prefix="1000,77,4096,16383,0,512,2047,9,129,8000,640,31,6001,15,333,12345",
             Hkv=8, D=128, bs=16, fused=False),
        # the prompts of a serving batch: 16 prompts of 1K to 16K tokens, v and k out of the fused projection
        dict(name="append prompts 1-16K", op="append",
             lens="1024,2047,3111,4096,5000,6143,7001,8192,9215,10240,11111,12288,13001,14336,15359,16384",
             prefix="0*16", Hkv=8, D=128, bs=16, fused=True),
        # the demo tree's accepted path
        dict(name="commit demo tree", op="commit", prefix="16", N=5, Hkv=2, D=64, bs=16, depth=2),
        # 64 sequences of 64-node trees, up to eight accepted drafts each
        dict(name="commit batch 64", op="commit", prefix="2048*64", N=64, Hkv=8, D=128, bs=16, depth=8),
        # the five-node demo tree on 16 tokens: the smallest call
        dict(name="attn demo tree", op="attn", prefix="16", N=5, Hq=2, Hkv=2, D=64, bs=16, depth=2, hot=0.0),
        # plain decoding (a tree of the root alone) for 32 sequences of odd lengths, one of them new
        dict(name="attn one node", op="attn",
             prefix="0,1,17,130,255,511,700,1001,1300,1537,2000,2222,2500,2999,3333,3700,4001,4096,4444,4800,5003,5500,5901,6144,6500,7000,7123,7400,7777,8000,8100,8191",
             N=1, Hq=32, Hkv=8, D=128, bs=64, depth=0, hot=0.01),
        # batched serving: 16 sequences, 26-node trees, 1K to 16K tokens in 16-token blocks: bound by reading the cache
        dict(name="attn batch 16, 1-16K", op="attn",
             prefix="1024,2047,3111,4096,5000,6143,7001,8192,9215,10240,11111,12288,13001,14336,15359,16384",
             N=26, Hq=32, Hkv=8, D=128, bs=16, depth=5, hot=0.01),
        # the 70B-shaped layer: 64 sequences of 8K tokens, 64 nodes, 8 query heads to a KV head: bound by the products
        dict(name="attn batch 64, 8K", op="attn", prefix="8192*64", N=64, Hq=64, Hkv=8, D=128, bs=16, depth=8, hot=0.0),
        # long prefixes: 4 sequences of 128K tokens, 192 nodes, a hundredth of the keys hot
        dict(name="attn 128K, 192 nodes", op="attn", prefix="131072*4", N=192, Hq=32, Hkv=8, D=128, bs=64, depth=10, hot=0.01),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "commit", "attn", "attn"])
    D = rng.choice([64, 128, 128])
    G = rng.choice([1, 2, 4, 8, 16])
    bs = rng.choice([16, 16, 32, 48, 64, 128, 144])
    if op == "rope":
        Hkv = rng.choice([1, 2, 3, 8])
        B, N = _log(rng, 1, 64), rng.randint(1, 256)
        while B * N * Hkv * G * D > 64 * 64 * 64 * 128:
            B, N = max(1, B // 2), max(1, N // 2)
        scaling = rng.choice(["none", "linear", "ntk", "bands"])
        return dict(op=op, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, rotary=rng.choice([D, D, D // 2, 32, 20, 10]),
                    interleaved=rng.random() < 0.5, fused=rng.random() < 0.5, theta=rng.choice([10000.0, 500000.0]),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                    low=1.0, high=rng.choice([4.0, 32.0]), orig=rng.choice([4096, 8192]),
                    mscale=1.0 if scaling != "bands" else rng.choice([1.0, 1.2]), start=_log(rng, 1, 1 << 20))
    if op == "append":
        B = _log(rng, 1, 32)
        lens = [0 if rng.random() < 0.1 else _log(rng, 1, 16384) for _ in range(B)]
        while sum(lens) > 130000:
            lens = [n // 2 for n in lens]
        if not any(lens):
            lens[0] = 1
        return dict(op=op, lens=",".join(map(str, lens)), prefix=",".join(str(rng.choice([0, _log(rng, 1, 2000)])) for _ in lens),
                    Hkv=rng.choice([1, 2, 5, 8]), D=D, bs=bs, fused=rng.random() < 0.5)
    if op == "commit":
        B = _log(rng, 1, 96)
        N = rng.randint(1, 256)
        return dict(op=op, prefix=",".join(str(rng.choice([0, _log(rng, 1, 2000)])) for _ in range(B)), N=N,
                    Hkv=rng.choice([1, 2, 5, 8]), D=D, bs=bs, depth=min(N - 1, rng.randint(0, 12)))
    Hkv = rng.choice([1, 2, 3, 8])
    N = rng.choice([1, _log(rng, 1, 256), rng.randint(1, 256)])
    B = _log(rng, 1, 48)
    top = _log(rng, 64, 65536)
    plens = [0 if rng.random() < 0.05 else _log(rng, max(1, top // 16), top) for _ in range(B)]
    while N * Hkv * G * sum(plens) > 4 * 192 * 32 * 131072 // 4 or sum(plens) * Hkv > 131072 * 8 * 2:
        plens = [p // 2 for p in plens]
    return dict(op=op, prefix=",".join(map(str, plens)), N=N, Hq=Hkv * G, Hkv=Hkv, D=D, bs=bs,
                depth=min(N - 1, rng.randint(0, 12)), hot=rng.choice([0.0, 0.01]))


def _lens(text):
    out = []
    for part in text.split(","):
        n, _, times = part.partition("*")
        out += [int(n)] * (int(times) if times else 1)
    return out


# ------------------------------------------------------------------------------------------------------------ inputs

def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _trees(case, B, seed):
    """Random trees of N nodes and the given depth, level by level: parents [B, N] and depths [B, N]."""
    N, top = case["N"], min(case.get("depth", 0), case["N"] - 1)
    r = np.random.default_rng([seed, 7])
    lv = np.zeros((B, N), np.int64)
    if N > 1:
        if top < 1:
            top = 1
        lv[:, 1:1 + top] = np.arange(1, top + 1)
        lv[:, 1 + top:] = r.integers(1, top + 1, (B, N - 1 - top))
        lv.sort(axis=1)
    parent = np.full((B, N), -1, np.int32)
    for b in range(B):
        first = np.searchsorted(lv[b], np.arange(top + 2))
        for i in range(1, N):
            d = lv[b, i]
            parent[b, i] = r.integers(first[d - 1], first[d])
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


def _pool(g, blocks, Hkv, bs, D, hot=0.0):
    """A pool of quantised rows: codes [blocks, Hkv, bs, D] and scale bytes [blocks, Hkv, bs]."""
    x = torch.randn((blocks, Hkv, bs, D), generator=g, device="cuda", dtype=torch.float32)
    if hot:
        x *= torch.where(torch.rand((blocks, Hkv, bs, 1), generator=g, device="cuda") < hot, 8.0, 1.0)
    return _quantise(x.to(torch.bfloat16).float())


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
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    D, Hkv = case["D"], case["Hkv"]
    s = dict(case=case)
    if case["op"] == "rope":
        B, N, Hq = case["B"], case["N"], case["Hq"]
        if case["fused"]:  # views of the projection's output: [q heads | k heads | v heads] of every token
            x = _normal(g, (B, N, Hq + 2 * Hkv, D))
            s["q"], s["k"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = _normal(g, (B, N, Hq, D)), _normal(g, (B, N, Hkv, D))
        r = np.random.default_rng([seed, 3])
        first = r.integers(case["start"], case["start"] + 64, (B, 1))
        s["pos"] = _i32(first + np.sort(r.integers(0, 11, (B, N)), axis=1))
        s["q_out"] = torch.empty((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty((B, N, Hkv, D), dtype=torch.bfloat16, device="cuda")
        return s
    plens, bs = _lens(case["prefix"]), case["bs"]
    B = len(plens)
    s["prefix_len"], s["prefix_len_host"] = _i32(plens), np.array(plens, np.int32)
    if case["op"] == "attn":
        N, Hq = case["N"], case["Hq"]
        s["table"], blocks = _paging(plens, bs, seed)
        s["k_cache"], ks = _pool(g, blocks, Hkv, bs, D, case["hot"])
        s["v_cache"], vs = _pool(g, blocks, Hkv, bs, D)
        s["scales"] = torch.stack((ks, vs), dim=-1).contiguous()
        s["q"] = _normal(g, (B, N, Hq, D))
        s["k_tree"], s["v_tree"] = _normal(g, (B, N, Hkv, D)), _normal(g, (B, N, Hkv, D))
        parent, depth = _trees(case, B, seed)
        s["mask"] = _masks(parent)
        s["pos"] = s["prefix_len"][:, None] + torch.from_numpy(depth).cuda()
        s["out"] = torch.empty((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, N, Hq), dtype=torch.float32, device="cuda")
        s["status"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "append":
        lens = _lens(case["lens"])
        T = sum(lens)
        s["cu_len"] = _i32(np.concatenate(([0], np.cumsum(lens))))
        if case["fused"]:
            x = _normal(g, (T, 2 * Hkv, D))
            s["k"], s["v"] = x[:, :Hkv], x[:, Hkv:]
        else:
            s["k"], s["v"] = _normal(g, (T, Hkv, D)), _normal(g, (T, Hkv, D))
        more = lens
    else:
        N, top = case["N"], case["depth"]
        s["k"], s["v"] = _normal(g, (B, N, Hkv, D)), _normal(g, (B, N, Hkv, D))
        parent, depth = _trees(case, B, seed)
        r = np.random.default_rng([seed, 5])
        acc, length = np.full((B, top + 1), -1, np.int32), np.zeros(B, np.int32)
        for b in range(B):
            n = int(r.integers(0, N))
            while depth[b, n] > top:
                n = int(parent[b, n])
            length[b] = depth[b, n]
            while n >= 0:
                acc[b, depth[b, n]] = n
                n = int(parent[b, n])
        s["accepted"], s["accept_len"] = _i32(acc), _i32(length)
        more = [top + 1] * B
    s["table"], blocks = _paging([p + n for p, n in zip(plens, more)], bs, seed)
    s["k_cache"], ks = _pool(g, blocks, Hkv, bs, D)
    s["v_cache"], vs = _pool(g, blocks, Hkv, bs, D)
    s["scales"] = torch.stack((ks, vs), dim=-1).contiguous()
    s["new_len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["status"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------- plain forms

def _frequencies(case):
    """Radians a position for each of the R/2 pairs, in 64 bits."""
    R, theta, s = case["rotary"], case["theta"], case["factor"]
    if case["scaling"] == "ntk" and R > 2:
        theta = theta * s ** (R / (R - 2))
    f = theta ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "bands":
        turns = case["orig"] * f / (2 * math.pi)  # rotations within the original context
        keep = ((turns - case["low"]) / (case["high"] - case["low"])).clamp(0, 1)
        f = keep * f + (1 - keep) * f / s
    return f


def _rope_plain(s):
    case = s["case"]
    R = case["rotary"]
    angle = s["pos"].double()[:, :, None, None] * _frequencies(case)  # 64 bits: far positions
    cos, sin = (angle.cos() * case["mscale"]).float(), (angle.sin() * case["mscale"]).float()

    def turn(x, out):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
        else:
            a, b = x[..., :R // 2], x[..., R // 2:R]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
        return out.copy_(torch.cat((y, x[..., R:]), dim=-1))

    return {"q": turn(s["q"], s["q_out"]), "k": turn(s["k"], s["k_out"])}


def _power(biased):
    """2^(biased - 127) in fp32, for biased in [1, 254], without rounding."""
    return (biased.int() << 23).view(torch.float32)


def _quantise(x):
    """Rows of fp32 values (the last axis) to e4m3 codes and scale bytes (see the top of the file)."""
    mant, exp = torch.frexp(x.abs().amax(dim=-1))  # mant in [0.5, 1)
    byte = torch.where(mant > 0, exp - 9 + (mant > 0.875) + 127, 1).clamp(1, 247)
    codes = (x * _power(254 - byte)[..., None]).clamp(-448, 448).to(F8)
    return codes, byte.to(torch.uint8)


def _write_plain(s, seq, token, k, v):
    """Rows k, v [n, Hkv, D] become tokens token[n] of sequences seq[n]."""
    bs = s["case"]["bs"]
    blk, row = s["table"][seq, token // bs].long(), token % bs
    for x, cache, which in ((k, "k_cache", 0), (v, "v_cache", 1)):
        codes, byte = _quantise(x.float())
        s[cache].view(torch.uint8)[blk, :, row] = codes.view(torch.uint8)
        s["scales"][blk, :, row, which] = byte
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "scales": s["scales"], "new_len": s["new_len"]}


def _append_plain(s):
    n = torch.arange(s["k"].shape[0], device="cuda")
    seq = torch.searchsorted(s["cu_len"][1:].contiguous(), n.int(), right=True)
    s["new_len"].copy_(s["prefix_len"] + s["cu_len"].diff())
    return _write_plain(s, seq, s["prefix_len"][seq] + n - s["cu_len"][seq], s["k"], s["v"])


def _commit_plain(s):
    step = torch.arange(s["accepted"].shape[1], device="cuda")
    seq, d = (step[None, :] <= s["accept_len"][:, None]).nonzero(as_tuple=True)
    node = s["accepted"][seq, d].long()
    s["new_len"].copy_(s["prefix_len"] + s["accept_len"] + 1)
    return _write_plain(s, seq, s["prefix_len"][seq] + d, s["k"][seq, node], s["v"][seq, node])


def _attn_plain(s):
    case = s["case"]
    N, Hkv, D, bs = case["N"], case["Hkv"], case["D"], case["bs"]
    B, G = s["q"].shape[0], case["Hq"] // case["Hkv"]
    t = torch.arange(max(1, int(s["prefix_len_host"].max())), device="cuda")
    blk, row = s["table"][:, t // bs].clamp(min=0).long(), t % bs

    def rows(cache, which):  # the prefix rows of every sequence, [B, Hkv, P, D]
        codes = s[cache].view(torch.uint8)[blk, :, row].view(F8).float()
        return (codes * _power(s["scales"][blk, :, row, which])[..., None]).transpose(1, 2)

    q = s["q"].float().view(B, N, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, N * G, D) * D ** -0.5
    far = q @ rows("k_cache", 0).transpose(2, 3)
    far.masked_fill_((t[None, :] >= s["prefix_len"][:, None])[:, None, None], -math.inf)
    near = q @ s["k_tree"].float().permute(0, 2, 3, 1)
    j = torch.arange(N, device="cuda")
    seen = (s["mask"][:, :, j // 64] >> (j % 64)) & 1
    near.masked_fill_((seen == 0).repeat_interleave(G, dim=1)[:, None], -math.inf)
    top = torch.maximum(far.amax(dim=-1), near.amax(dim=-1))[..., None]
    far, near = far.sub_(top).exp_(), near.sub_(top).exp_()
    total = far.sum(dim=-1, keepdim=True) + near.sum(dim=-1, keepdim=True)
    o = (far @ rows("v_cache", 1) + near @ s["v_tree"].float().transpose(1, 2)) / total
    lse = (top + total.log()).squeeze(-1)
    s["out"].copy_(o.view(B, Hkv, N, G, D).transpose(1, 2).reshape(B, N, Hkv * G, D))
    s["lse"].copy_(lse.view(B, Hkv, N, G).transpose(1, 2).reshape(B, N, Hkv * G))
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------------------------------------- the library's calls

def _run_own(s):
    import tree_attention_speculative_gb300 as ts
    case = s["case"]
    if case["op"] == "rope":
        if "rope" not in s:  # kept by the program, as its model's configuration is
            s["rope"] = ts.RopeConfig(theta=case["theta"], rotary_dim=case["rotary"], interleaved=case["interleaved"],
                                      scaling=case["scaling"], factor=case["factor"], low_rot=case["low"],
                                      high_rot=case["high"], orig_len=case["orig"], mscale=case["mscale"])
        ts.tree_rope(s["q"], s["k"], s["pos"], s["q_out"], s["k_out"], s["rope"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if case["op"] == "attn":
        p = ts.attn_params(s["q"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], s["prefix_len_host"],
                           s["k_tree"], s["v_tree"], s["mask"], s["pos"], s["out"], s["lse"], s["status"])
        if "workspace" not in s:  # zero-filled once, kept by the program
            s["workspace"] = torch.zeros(ts.tree_attn_q8_workspace_size(p), dtype=torch.uint8, device="cuda")
        ts.tree_attn_fwd_q8(p, s["scales"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "append":
        ts.tree_cache_append_q8(s["k"], s["v"], s["cu_len"], s["prefix_len"], s["k_cache"], s["v_cache"], s["scales"],
                                s["table"], s["new_len"], s["status"])
    else:
        ts.tree_commit_accepted_q8(s["k"], s["v"], s["accepted"], s["accept_len"], s["prefix_len"], s["k_cache"],
                                   s["v_cache"], s["scales"], s["table"], s["new_len"], s["status"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "scales": s["scales"], "new_len": s["new_len"]}


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope_plain, "append": _append_plain, "commit": _commit_plain, "attn": _attn_plain}[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "rope":
        values = case["B"] * case["N"] * (case["Hq"] + Hkv) * D
        return {"bytes": 4 * values + 4 * case["B"] * case["N"], "flops": 3 * values * case["rotary"] // D}
    plens = _lens(case["prefix"])
    B = len(plens)
    if case["op"] == "attn":
        N, Hq = case["N"], case["Hq"]
        cache = sum(plens) * Hkv * (2 * D + 2) + 4 * sum(-(-p // case["bs"]) for p in plens)
        tree = B * N * (2 * Hkv * D * 2 + 8 * ((N + 63) // 64))
        return {"bytes": cache + tree + B * N * Hq * (4 * D + 4), "flops": 4 * D * Hq * N * (sum(plens) + B * (case["depth"] // 2 + 1))}
    if case["op"] == "append":
        rows = sum(_lens(case["lens"])) * Hkv * 2
    else:
        rows = B * (case["depth"] // 2 + 1) * Hkv * 2  # about half the depth is accepted
    return {"bytes": rows * (3 * D + 1) + 24 * B, "flops": 3 * rows * D}


# ------------------------------------------------------------------------------------------ the definitions in 64 bits

def _two_to(e):
    """2^e as doubles, exactly, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest_e4m3(x):
    """The e4m3 value next to x (a double within +-448), ties to the even code."""
    _, e = torch.frexp(x)
    step = (e - 4).clamp(min=-9)  # the codes around x are 2^step apart
    return torch.round(x * _two_to(-step)) * _two_to(step)  # torch.round: halves to even


def _exact_rows(s, jobs, new_len):
    """The caches after each (sequence, first token, k rows, v rows) of jobs is written."""
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    scales, bs = s["scales"].clone(), s["case"]["bs"]
    for b, first, k, v in jobs:
        for x, cache, which in ((k, k_cache, 0), (v, v_cache, 1)):
            if not x.shape[0]:
                continue
            x = x.double()
            largest = x.abs().amax(dim=-1, keepdim=True)
            e = torch.ceil(torch.log2(largest / 448)).clamp(min=-126)  # smallest power of two that fits ...
            e = torch.where(448 * _two_to(e - 1) >= largest, e - 1, e)  # ... whatever log2 rounds to
            e = torch.where(448 * _two_to(e) < largest, e + 1, e).clamp(min=-126)
            y = _nearest_e4m3(x * _two_to(-e))
            t = torch.arange(first, first + x.shape[0], device="cuda")
            blk = s["table"][b].long()[t // bs]
            cache[blk, :, t % bs] = y
            scales[blk, :, t % bs, which] = (e.squeeze(-1) + 127).to(torch.uint8)
    return {"k_cache": k_cache, "v_cache": v_cache, "scales": scales, "new_len": new_len}


def exact(case, seed):
    s = prepare(case, seed)
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "rope":
        R, s_ = case["rotary"], case["factor"]
        theta = case["theta"] * (s_ ** (R / (R - 2)) if case["scaling"] == "ntk" and R > 2 else 1.0)
        freq = []
        for i in range(R // 2):
            f = math.exp(-2 * i / R * math.log(theta))
            if case["scaling"] == "linear":
                f /= s_
            elif case["scaling"] == "bands":
                g = (case["orig"] / (2 * math.pi / f) - case["low"]) / (case["high"] - case["low"])
                f = f if g >= 1 else f / s_ if g <= 0 else g * f + (1 - g) * f / s_
            freq.append(f)
        angle = s["pos"].double()[:, :, None, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
        unit = torch.polar(torch.full_like(angle, case["mscale"]), angle)
        done = {}
        for name in ("q", "k"):
            x = s[name].double().clone()
            pairs = x[..., :R].unflatten(-1, (R // 2, 2)) if case["interleaved"] else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
            x[..., :R] = (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)
            done[name] = x
        return done
    plens, bs = _lens(case["prefix"]), case["bs"]
    if case["op"] == "append":
        cu = s["cu_len"].tolist()
        jobs = [(b, p, s["k"][cu[b]:cu[b + 1]], s["v"][cu[b]:cu[b + 1]]) for b, p in enumerate(plens)]
        return _exact_rows(s, jobs, _i32([p + cu[b + 1] - cu[b] for b, p in enumerate(plens)]))
    if case["op"] == "commit":
        jobs, new = [], []
        for b, p in enumerate(plens):
            path = s["accepted"][b, :int(s["accept_len"][b]) + 1].long()
            jobs.append((b, p, s["k"][b, path], s["v"][b, path]))
            new.append(p + len(path))
        return _exact_rows(s, jobs, _i32(new))
    N, Hq = case["N"], case["Hq"]
    G = Hq // Hkv
    out = torch.empty((len(plens), N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((len(plens), N, Hq), dtype=torch.float64, device="cuda")
    for b, p in enumerate(plens):
        bits = s["mask"][b].cpu().numpy().view(np.uint8).reshape(N, -1)
        seen = torch.from_numpy(np.unpackbits(bits, axis=1, bitorder="little")[:, :N].astype(bool)).cuda()
        blocks = s["table"][b, :-(-p // bs)].long()
        for g in range(Hkv):
            keys, values = [], []
            for cache, which, tree, into in (("k_cache", 0, "k_tree", keys), ("v_cache", 1, "v_tree", values)):
                c = s[cache].view(torch.uint8)[blocks, g].view(F8).double()
                e = s["scales"][blocks, g, :, which].double() - 127
                into += [(c * torch.pow(2.0, e)[..., None]).reshape(-1, D)[:p], s[tree][b, :, g].double()]
            keys, values = torch.cat(keys), torch.cat(values)
            allowed = torch.cat((torch.ones((N, p), dtype=torch.bool, device="cuda"), seen), dim=1)
            for h in range(g * G, (g + 1) * G):
                logits = (s["q"][b, :, h].double() @ keys.T) / math.sqrt(D)
                logits = torch.where(allowed, logits, torch.full_like(logits, -math.inf))
                lse[b, :, h] = torch.logsumexp(logits, dim=1)
                out[b, :, h] = torch.exp(logits - lse[b, :, h, None]) @ values
    return {"out": out, "lse": lse}
