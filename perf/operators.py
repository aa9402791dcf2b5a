"""Decode operators over a quantised, block-selected or drafted K/V cache: their cases, plain forms and exact values.

Three families, all over a cache [B, Hkv, Ncap, d] of which a sequence uses its first len keys:

* quant: rows quantised to 8 bits as they are written (int8: scale = amax / 127; e4m3: the smallest power of two
  that brings the row under 448), read back, and the attention that reads them (all keys, or listed ones);
* block: per-block minima and maxima of the keys, blocks chosen by the upper bound of q.k that they give (summed over
  the group's query heads), and the attention over the chosen blocks;
* tree: T drafted tokens of a sequence attend to its cache and to one another under a bit mask.
"""

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
CODE_TYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the prompt of one sequence goes into an int8 cache, from the projection's token-major rows, and is read back
        {"name": "write_prompt_int8", "op": "write", "B": 1, "Hkv": 8, "d": 128, "n": 32768, "fmt": "int8"},
        # three short ragged prompts into an e4m3 cache of 64-channel heads
        {"name": "write_ragged_e4m3", "op": "write", "B": 3, "Hkv": 8, "d": 64, "n": 1001, "fmt": "e4m3"},
        # one token of a short chat: quantise the new row, attend over all 4097
        {"name": "step_int8_n4k", "op": "qstep", "B": 1, "Hkv": 8, "G": 4, "d": 64, "N": 4097, "fmt": "int8"},
        # dense decode at the Llama-3.1-8B-like shape, 8 bits instead of 16
        {"name": "decode_int8_n100k", "op": "qstep", "B": 4, "Hkv": 8, "G": 4, "d": 128, "N": 102400, "fmt": "int8"},
        # the attention of a SOCKET step at that shape: 3103 listed keys of each pair
        {"name": "listed_e4m3_k3103", "op": "qlist", "B": 4, "Hkv": 8, "G": 4, "d": 128, "N": 102400, "k": 3103, "fmt": "e4m3"},
        # summaries of a prompt of that shape
        {"name": "summarize_n100k", "op": "summarize", "B": 4, "Hkv": 8, "d": 128, "N": 102400, "block": 32},
        # one token at the Llama-3.2-1B-like shape: refresh the last block, choose 62 of 2048 blocks, attend
        {"name": "block_step_n32k", "op": "bstep", "B": 1, "Hkv": 8, "G": 4, "d": 64, "N": 32768, "block": 16, "k": 62, "kv": "bf16"},
        # the same at the Llama-3.1-8B-like shape: 97 blocks of 32, about the keys that its top-k keeps
        {"name": "block_step_n100k", "op": "bstep", "B": 4, "Hkv": 8, "G": 4, "d": 128, "N": 102400, "block": 32, "k": 97, "kv": "bf16"},
        # a chain of 5 drafted tokens on a short cache
        {"name": "tree_t5_n4k", "op": "tree", "B": 1, "Hkv": 8, "G": 4, "d": 64, "N": 4099, "T": 5, "kv": "bf16", "out": "f32"},
        # 16 drafted tokens at the Llama-3.1-8B-like shape
        {"name": "tree_t16_n100k", "op": "tree", "B": 4, "Hkv": 8, "G": 4, "d": 128, "N": 102384, "T": 16, "kv": "bf16", "out": "f32"},
        # a wide tree, ragged sequences
        {"name": "tree_t64_n100k", "op": "tree", "B": 4, "Hkv": 8, "G": 4, "d": 128, "N": 102336, "T": 64, "kv": "bf16", "out": "bf16"},
        # drafted tokens over an int8 cache with 8 query heads to a KV head (Qwen3-30B-like heads)
        {"name": "tree_t7_int8_n32k", "op": "tree", "B": 2, "Hkv": 4, "G": 8, "d": 128, "N": 32761, "T": 7, "kv": "int8", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "qstep", "qstep", "qlist", "summarize", "bstep", "bstep", "tree", "tree", "tree"])
    c = {"op": op, "B": _log(rng, 1, 8), "Hkv": rng.choice([1, 2, 3, 4, 8]), "d": rng.choice([64, 128])}
    most = 4 * 8 * 102400 * 128 // (c["B"] * c["Hkv"] * c["d"])    # keys that cost what the largest listed case does
    if op == "write":
        c["n"], c["fmt"] = _log(rng, 1, min(32768, most)), rng.choice(["int8", "e4m3"])
        return c
    c["N"] = _log(rng, 16, min(131072, most))
    if op == "summarize":
        c["block"] = rng.choice([16, 32, 64])
        return c
    c["G"] = rng.choice([1, 2, 4, 5, 7, 8])
    if op in ("qstep", "qlist"):
        c["fmt"] = rng.choice(["int8", "e4m3"])
        if op == "qlist":
            c["k"] = _log(rng, 1, min(c["N"], 8192))
    elif op == "bstep":
        c["block"], c["kv"] = rng.choice([16, 32, 64]), rng.choice(["bf16", "int8", "e4m3"])
        c["k"] = _log(rng, 2, 128)
    else:
        c["T"], c["kv"], c["out"] = _log(rng, 1, 64), rng.choice(["bf16", "bf16", "int8", "e4m3"]), rng.choice(["f32", "bf16"])
        c["N"] = max(1, min(c["N"], 4 * 8 * 64 * 4 * 102336 // (c["B"] * c["Hkv"] * c["T"] * c["G"])))
    return c


# ---------------------------------------------------------------- inputs
def _quantise(x, fmt):
    """f32 rows -> (codes, scales [..., 1])."""
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "int8":
        s = amax / torch.full_like(amax, 127.0)
        # in 64 bits: a quotient next to a half would round twice in 32
        c = torch.where(s > 0, (x.to(F64) / s.to(F64)).round(), 0.0)
        return c.clamp(-127, 127).to(torch.int8), s
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)      # amax = m 2^e <= 448 2^e', 448 = 0.875 2^9
    s = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), 0.0)
    c = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0)
    return c.to(torch.float8_e4m3fn), s


def _values(codes, scales):
    return codes.to(F32) * scales


def _cdiv(a, b):
    return -(-a // b)


def _lens(c):
    """The sequences of a batch differ in length: N keys down to about half of them."""
    return [max(1, c["N"] - b * c["N"] // (2 * c["B"])) for b in range(c["B"])]


def _rows(gen, B, Hkv, n, d, spread):
    """bf16 rows with 4 channels of each head 8 times as large and, for spread > 0, lognormal norms."""
    x = torch.randn(B, Hkv, n, d, generator=gen, device="cuda")
    ch = torch.rand(Hkv, d, generator=gen, device="cuda").argsort(-1)[:, :4]
    x *= torch.ones(Hkv, d, device="cuda").scatter_(1, ch, 8.0)[None, :, None]
    if spread > 0:
        x *= torch.exp(spread * torch.randn(B, Hkv, n, 1, generator=gen, device="cuda"))
    return x.to(BF16)


def _ancestors(gen, B, T):
    """[B, T, T] bool: token t of a random tree sees itself and the tokens on its way to the root."""
    parent = [torch.randint(-1, t, (B,), generator=gen, device="cuda") if t else torch.full((B,), -1, device="cuda") for t in range(T)]
    a, rows = torch.zeros(B, T, T, dtype=torch.bool, device="cuda"), torch.arange(B, device="cuda")
    for t in range(T):
        a[:, t] = a[rows, parent[t].clamp(min=0)] & (parent[t] >= 0)[:, None]
        a[:, t, t] = True
    return a


def _pack(seen):
    """[B, T, T] bool -> [B, T, ceil(T / 32)] int32, bit j % 32 of word j / 32 for drafted key j."""
    B, T, _ = seen.shape
    bits = torch.nn.functional.pad(seen, (0, _cdiv(T, 32) * 32 - T)).view(B, T, -1, 32).long()
    w = (bits << torch.arange(32, device=seen.device)).sum(-1)
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32).contiguous()


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    s = {"case": c}
    if c["op"] == "write":
        n = c["n"]
        # as a projection leaves them: [B, n, Hkv, d], seen as [B, Hkv, n, d]
        s["K"], s["V"] = (_rows(gen, B, Hkv, n, d, sp).transpose(1, 2).contiguous().transpose(1, 2) for sp in (0.0, 0.5))
        cap = _cdiv(n, 32) * 32
        s["Kq"], s["Vq"] = (torch.zeros(B, Hkv, cap, d, device="cuda").to(CODE_TYPE[c["fmt"]]) for _ in range(2))
        s["scales"] = torch.zeros(B, Hkv, cap, 2, device="cuda")
        s["Kr"], s["Vr"] = torch.empty(B, Hkv, n, d, dtype=BF16, device="cuda"), torch.empty(B, Hkv, n, d, dtype=BF16, device="cuda")
        return s
    T, N = c.get("T", 1), c["N"]
    drafts = T if c["op"] == "tree" else 0
    cap = _cdiv(N + drafts, 64) * 64
    K, V = _rows(gen, B, Hkv, cap, d, 0.0), _rows(gen, B, Hkv, cap, d, 0.5)
    if c["op"] == "summarize":
        s["K"] = K
        s["bsum"] = torch.zeros(B, Hkv, _cdiv(cap, c["block"]), 2, d, dtype=BF16, device="cuda")
        return s
    G = c["G"]
    Hq = Hkv * G
    Q = torch.randn(B, T, Hq, d, generator=gen, device="cuda").to(BF16)
    # some keys point along a query of their group: they carry most of the weight
    q = Q[:, 0].float().view(B, Hkv, G, d)[:, :, 0]
    at = torch.randint(0, N, (B, Hkv, 16), generator=gen, device="cuda")[..., None].expand(B, Hkv, 16, d)
    needle = torch.randn(B, Hkv, 16, d, generator=gen, device="cuda") + 2.0 * (math.sqrt(d) * q / q.norm(dim=-1, keepdim=True))[:, :, None]
    K.scatter_(2, at, needle.to(BF16))
    s["Q"] = Q if drafts else Q[:, 0].contiguous()
    s["scale"] = 1.0 / math.sqrt(d)
    lens = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
    s["lens"] = lens
    last = (lens.long() - 1)[:, None, None, None]
    fmt = c.get("fmt") or c["kv"]
    s["scales"] = None
    if fmt != "bf16":
        if c["op"] == "qstep":      # the newest token's row, to be quantised by the step
            s["Kn"], s["Vn"] = (x.gather(2, last.expand(B, Hkv, 1, d)) for x in (K, V))
            K.scatter_(2, last.expand(B, Hkv, 1, d), 0.0)
            V.scatter_(2, last.expand(B, Hkv, 1, d), 0.0)
            s["starts"] = lens - 1
        (kc, ks), (vc, vs) = _quantise(K.float(), fmt), _quantise(V.float(), fmt)
        s["scales"] = torch.cat((ks, vs), -1).contiguous()
        s["K"], s["V"] = kc, vc
    else:
        s["K"], s["V"] = K, V
    if c["op"] == "qlist":
        s["idx"] = torch.rand(B, Hkv, N, generator=gen, device="cuda").argsort(-1)[..., : c["k"]].sort(-1)[0].to(torch.int32)
    if c["op"] == "bstep":
        bl = c["block"]
        live = (torch.arange(cap, device="cuda") < last[:, :, 0])[:, :, :, None]     # before the newest token
        keys = K.float() if fmt == "bf16" else _values(s["K"], s["scales"][..., :1])
        mn = _outward(keys.masked_fill(~live, math.inf).view(B, Hkv, cap // bl, bl, d).amin(3), -1)
        mx = _outward(keys.masked_fill(~live, -math.inf).view(B, Hkv, cap // bl, bl, d).amax(3), 1)
        s["bsum"] = torch.stack((mn, mx), 3).masked_fill(~live.view(B, 1, -1, bl)[:, :, :, 0][..., None, None], 0.0).contiguous()
        s["starts"] = lens - 1
        s["idx"] = torch.empty(B, Hkv, c["k"], dtype=torch.int32, device="cuda")
    if drafts:
        s["seen"] = _ancestors(gen, B, T)
        s["mask"] = _pack(s["seen"])
    s["O"] = torch.empty(s["Q"].shape, dtype=BF16 if c.get("out") == "bf16" else F32, device="cuda")
    return s


def _outward(x, sign):
    """bf16 of f32 x, rounded down (sign -1) or up (sign 1)."""
    r = x.to(BF16)
    bits = r.view(torch.int16).int()
    wrong = (r.float() > x) if sign < 0 else (r.float() < x)
    step = torch.where((bits < 0) == (sign < 0), 1, -1)             # away from zero or towards it
    return torch.where(wrong, (bits + step).to(torch.int16), bits.to(torch.int16)).view(BF16)


# ---------------------------------------------------------------- plain forms
def _attend(Q, K, V, seen, scale):
    """Q [B, Hkv, R, d], K and V [B, Hkv, n, d] in 32 bits, seen [B, 1 or Hkv, 1 or R, n]: softmax attention, 0 where nothing is seen."""
    x = (Q @ K.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    return (p @ V) / p.sum(-1, keepdim=True).clamp(min=1e-37)


def _group(Q, Hkv):
    """[B, T, Hq, d] or [B, Hq, d] -> [B, Hkv, T * G, d] in 32 bits."""
    Q = Q if Q.dim() == 4 else Q[:, None]
    B, T, Hq, d = Q.shape
    return Q.float().view(B, T, Hkv, Hq // Hkv, d).transpose(1, 2).reshape(B, Hkv, -1, d)


def _cache(s):
    if s["scales"] is None:
        return s["K"].float(), s["V"].float()
    return _values(s["K"], s["scales"][..., :1]), _values(s["V"], s["scales"][..., 1:])


def _plain_blocks(s):
    """The step's summary of the newest token's block, the chosen blocks (ascending, then -1), and the attention."""
    c, lens = s["case"], s["lens"].long()
    B, Hkv, d, bl, k = c["B"], c["Hkv"], c["d"], c["block"], c["k"]
    b, h = torch.arange(B, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[None, :, None]
    last = (lens - 1) // bl
    rows = (last * bl)[:, None, None] + torch.arange(bl, device="cuda")
    keys = s["K"][b, h, rows]
    keys = keys.float() if s["scales"] is None else _values(keys, s["scales"][b, h, rows][..., :1])
    live = (rows < lens[:, None, None])[..., None]
    mn, mx = keys.masked_fill(~live, math.inf).amin(2), keys.masked_fill(~live, -math.inf).amax(2)
    s["bsum"][b[..., 0], h[..., 0], last[:, None]] = torch.stack((_outward(mn, -1), _outward(mx, 1)), 2)
    q = s["Q"].view(B, Hkv, -1, d).to(F64)
    t = torch.cat((q.clamp(max=0).sum(2), q.clamp(min=0).sum(2)), -1)
    nb = (lens + bl - 1) // bl
    NB = int(s["bsum"].shape[2])
    score = (s["bsum"].view(B, Hkv, NB, 2 * d).to(F64) @ t[..., None])[..., 0].to(F32)     # 64 bits: near ties
    j = torch.arange(NB, device="cuda")
    here = j < nb[:, None, None]
    forced = (j == 0) | (j == nb[:, None, None] - 1)
    key = score.masked_fill(forced, math.inf).masked_fill(~here, -math.inf)
    top = key.sort(dim=-1, descending=True, stable=True)[1][..., :k]
    top = torch.nn.functional.pad(top, (0, k - top.shape[-1]), value=NB)
    top = torch.where(top < nb[:, None, None], top, NB).sort(-1)[0]
    idx = torch.where(top < NB, top, -1).to(torch.int32)
    rows = (top[..., None] * bl + torch.arange(bl, device="cuda")).flatten(2)
    seen = (rows < lens[:, None, None]) & (top < NB).repeat_interleave(bl, -1)
    rows = rows.clamp(max=s["K"].shape[2] - 1)
    K, V = s["K"][b, h, rows], s["V"][b, h, rows]
    if s["scales"] is not None:
        sc = s["scales"][b, h, rows]
        K, V = _values(K, sc[..., :1]), _values(V, sc[..., 1:])
    O = _attend(_group(s["Q"], Hkv), K.float(), V.float(), seen[:, :, None], s["scale"])
    return {"O": O.reshape(s["Q"].shape), "idx": idx, "bsum": s["bsum"]}


def _plain(s):
    c = s["case"]
    op, B, Hkv, d = c["op"], c["B"], c["Hkv"], c["d"]
    if op == "write":
        (kc, ks), (vc, vs) = _quantise(s["K"].float(), c["fmt"]), _quantise(s["V"].float(), c["fmt"])
        return {"K": _values(kc, ks).to(BF16), "V": _values(vc, vs).to(BF16), "scales": torch.cat((ks, vs), -1)}
    if op == "summarize":
        N, bl = c["N"], c["block"]
        nb = _cdiv(N, bl)
        live = (torch.arange(nb * bl, device="cuda") < N)[:, None]
        K = s["K"][:, :, : nb * bl]
        mn = K.masked_fill(~live, math.inf).view(B, Hkv, nb, bl, d).amin(3)
        mx = K.masked_fill(~live, -math.inf).view(B, Hkv, nb, bl, d).amax(3)
        s["bsum"][:, :, :nb] = torch.stack((mn, mx), 3)
        return {"bsum": s["bsum"]}
    if op == "bstep":
        return _plain_blocks(s)
    if op == "qlist":
        rows = s["idx"].long()
        b, h = torch.arange(B, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[None, :, None]
        sc = s["scales"][b, h, rows]
        K, V = _values(s["K"][b, h, rows], sc[..., :1]), _values(s["V"][b, h, rows], sc[..., 1:])
        O = _attend(_group(s["Q"], Hkv), K, V, torch.ones(1, 1, 1, 1, dtype=torch.bool, device="cuda"), s["scale"])
        return {"O": O.view(s["Q"].shape)}
    if op == "qstep":
        b, h = torch.arange(B, device="cuda")[:, None], torch.arange(Hkv, device="cuda")[None]
        at = s["starts"].long()[:, None]
        (kc, ks), (vc, vs) = _quantise(s["Kn"].float(), c["fmt"]), _quantise(s["Vn"].float(), c["fmt"])
        s["K"].view(torch.uint8)[b, h, at], s["V"].view(torch.uint8)[b, h, at] = kc[:, :, 0].view(torch.uint8), vc[:, :, 0].view(torch.uint8)
        new = torch.cat((ks, vs), -1)[:, :, 0]
        s["scales"][b, h, at] = new
        K, V = _cache(s)
        seen = (torch.arange(K.shape[2], device="cuda") < s["lens"][:, None])[:, None, None]
        O = _attend(_group(s["Q"], Hkv), K, V, seen, s["scale"])
        return {"O": O.view(s["Q"].shape), "K": _values(kc, ks).to(BF16), "V": _values(vc, vs).to(BF16), "scales": s["scales"]}
    K, V = _cache(s)
    T, G = c["T"], c["G"]
    lens = s["lens"].long()[:, None, None]
    j = torch.arange(K.shape[2], device="cuda") - lens                      # [B, 1, n]: drafted key, < 0 in the cache
    seen = (j < 0) | ((j < T) & s["seen"].gather(2, j.clamp(0, T - 1).expand(B, T, -1)))
    seen = seen[:, :, None].expand(B, T, G, -1).reshape(B, 1, T * G, -1)
    O = _attend(_group(s["Q"], Hkv), K, V, seen, s["scale"])
    return {"O": O.view(B, Hkv, T, G, d).transpose(1, 2).reshape(s["Q"].shape).to(s["O"].dtype)}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from hash_scored_top_b200 import api

    c = s["case"]
    op, N = c["op"], c.get("N")
    if op == "write":
        api.quant_append(s["K"], s["V"], s["Kq"], s["Vq"], s["scales"])
        api.quant_read(s["Kq"], s["Vq"], s["scales"], s["Kr"], s["Vr"])
        return {"K": s["Kr"], "V": s["Vr"], "scales": s["scales"][:, :, : c["n"]]}
    if op == "summarize":
        api.block_summarize(s["K"], c["block"], s["bsum"], n_count=N)
        return {"bsum": s["bsum"]}
    if "ws" not in s:       # a program keeps its workspace
        Ncap, k = s["K"].shape[2], c.get("k", 0)
        what = {"qstep": api.OP_QUANT_DECODE, "qlist": api.OP_QUANT_SPARSE_ATTEND, "bstep": api.OP_BLOCK_DECODE, "tree": api.OP_TREE_DECODE}[op]
        size = api.workspace_bytes(what, c["B"], c["Hkv"] * c["G"], c["Hkv"], Ncap, N, c["d"], c.get("block", 0), 0, c.get("T", k))
        s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
        if op == "qstep":
            s["Kr"], s["Vr"] = torch.empty_like(s["Kn"]), torch.empty_like(s["Vn"])
    if op == "qstep":
        api.quant_append(s["Kn"], s["Vn"], s["K"], s["V"], s["scales"], starts=s["starts"])
        api.quant_decode(s["Q"], s["K"], s["V"], s["scales"], N, s["scale"], s["O"], lens=s["lens"], ws=s["ws"])
        api.quant_read(s["K"], s["V"], s["scales"], s["Kr"], s["Vr"], starts=s["starts"])
        return {"O": s["O"], "K": s["Kr"], "V": s["Vr"], "scales": s["scales"]}
    if op == "qlist":
        api.quant_sparse_attend(s["Q"], s["K"], s["V"], s["scales"], s["idx"], s["scale"], s["O"], ws=s["ws"])
        return {"O": s["O"]}
    if op == "bstep":
        api.block_summarize(s["K"], c["block"], s["bsum"], n_count=1, scales=s["scales"], starts=s["starts"], lens=s["lens"])
        api.block_decode(s["Q"], s["K"], s["V"], s["bsum"], N, c["block"], c["k"], 1, 1, s["scale"], s["O"], scales=s["scales"],
                         lens=s["lens"], idx_out=s["idx"], ws=s["ws"])
        return {"O": s["O"], "idx": s["idx"], "bsum": s["bsum"]}
    api.tree_decode(s["Q"], s["K"], s["V"], N, s["scale"], s["O"], mask=s["mask"], scales=s["scales"], lens=s["lens"], ws=s["ws"])
    return {"O": s["O"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    op, pairs, d = c["op"], c["B"] * c["Hkv"], c["d"]
    if op == "write":       # 16-bit rows in, codes and scales out; the same back
        return {"bytes": pairs * c["n"] * 2 * (4 * d + 2 * d + 8), "flops": pairs * c["n"] * 2 * 6 * d}
    N = c["N"]
    if op == "summarize":
        return {"bytes": pairs * (N * 2 * d + _cdiv(N, c["block"]) * 4 * d), "flops": pairs * N * 2 * d}
    G, T = c["G"], c.get("T", 1)
    heads = pairs * G * d
    keys = sum(_lens(c)) * c["Hkv"]
    row = 4 * d if (c.get("fmt") or c["kv"]) == "bf16" else 2 * d + 8
    if op == "qstep":
        return {"bytes": keys * row + heads * 6 + pairs * (4 * d + row) * 2, "flops": keys * 4 * d * G}
    if op == "qlist":
        return {"bytes": pairs * c["k"] * (row + 4) + heads * 6, "flops": pairs * c["k"] * 4 * d * G}
    if op == "bstep":
        read = sum(min(c["k"] * c["block"], n) for n in _lens(c)) * c["Hkv"]
        blocks = sum(_cdiv(n, c["block"]) for n in _lens(c)) * c["Hkv"]
        return {"bytes": blocks * 4 * d + read * row + heads * 6 + pairs * c["k"] * 4, "flops": blocks * 4 * d + read * 4 * d * G}
    keys += pairs * T
    return {"bytes": keys * row + heads * T * (4 if c["out"] == "bf16" else 6), "flops": keys * 4 * d * G * T}


# ---------------------------------------------------------------- exact values
def _exact_row_scale(x, fmt):
    """The scale's definition in 64 bits, rounded to the 32 that hold it."""
    a = x.abs().max(-1)[0]
    if fmt == "int8":
        return (a / 127).to(F32).to(F64)
    e = torch.ceil(torch.log2(a.clamp(min=1e-300) / 448)).clamp(min=-126)
    e = torch.where(torch.exp2(e - 1) * 448 >= a, e - 1, e).clamp(min=-126)       # a log2 just above a whole number
    return torch.where(a > 0, torch.exp2(e), 0.0)


def _exact_codes(x, s, fmt):
    y = torch.where(s[..., None] > 0, x / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    if fmt == "int8":
        return y.round().clamp(-127, 127)
    # e4m3: steps of 2^-3 of the value's power of two, 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
    return (y / step).round() * step


def _exact_softmax(q, k, v, seen, scale):
    x = (q @ k.T) * scale
    x = torch.where(seen, x, torch.tensor(-math.inf, dtype=F64, device=x.device))
    return torch.softmax(x, -1).nan_to_num(0.0) @ v


def exact(case, seed):
    s, c = prepare(case, seed), case
    op, B, Hkv, d = c["op"], c["B"], c["Hkv"], c["d"]
    if op in ("write", "qstep"):
        new = [s[k].to(F64) for k in (("K", "V") if op == "write" else ("Kn", "Vn"))]
        sc = [_exact_row_scale(x, c["fmt"]) for x in new]
        back = [_exact_codes(x, y, c["fmt"]) * y[..., None] for x, y in zip(new, sc)]
        if op == "write":
            return {"K": back[0], "V": back[1], "scales": torch.stack(sc, -1)}
    if op == "summarize":
        out = s["bsum"].to(F64)
        for j in range(_cdiv(c["N"], c["block"])):
            part = s["K"][:, :, j * c["block"] : min(c["N"], (j + 1) * c["block"])].to(F64)
            out[:, :, j, 0], out[:, :, j, 1] = part.min(2)[0], part.max(2)[0]
        return {"bsum": out}
    G, T = c["G"], c.get("T", 1)
    Q = s["Q"].to(F64).view(B, T, Hkv, G, d)
    O = torch.zeros(B, T, Hkv, G, d, dtype=F64, device="cuda")
    idx = bsum = None
    if op == "bstep":
        bsum, idx = s["bsum"].to(F64), torch.full((B, Hkv, c["k"]), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        n = int(s["lens"][b])
        for h in range(Hkv):
            k, v = s["K"][b, h].to(F64), s["V"][b, h].to(F64)
            if s["scales"] is not None:
                k, v = k * s["scales"][b, h, :, :1].to(F64), v * s["scales"][b, h, :, 1:].to(F64)
            q = Q[b, :, h].reshape(T * G, d)
            if op == "qstep":
                k[n - 1], v[n - 1] = back[0][b, h, 0], back[1][b, h, 0]
                s["scales"][b, h, n - 1] = torch.stack((sc[0][b, h, 0], sc[1][b, h, 0])).to(F32)
            if op == "qlist":
                rows = s["idx"][b, h].long()
                k, v = k[rows], v[rows]
                seen = torch.ones(1, len(rows), dtype=torch.bool, device="cuda")
            elif op == "tree":
                seen = torch.zeros(T, k.shape[0], dtype=torch.bool, device="cuda")
                seen[:, :n] = True
                seen[:, n : n + T] = s["seen"][b]
                seen = seen.repeat_interleave(G, 0)
            elif op == "bstep":
                bl, nb = c["block"], _cdiv(n, c["block"])
                tail = k[(nb - 1) * bl : n]
                lo, hi = tail.min(0)[0], tail.max(0)[0]
                bsum[b, h, nb - 1] = torch.stack((_outward(lo.to(F32), -1), _outward(hi.to(F32), 1))).to(F64)
                bound = torch.maximum(q[:, None] * bsum[b, h, None, :nb, 0], q[:, None] * bsum[b, h, None, :nb, 1]).sum((0, 2)).to(F32)
                order = sorted(range(nb), key=lambda j, t=bound.tolist(): (j not in (0, nb - 1), -t[j], j))
                chosen = sorted(order[: c["k"]])
                idx[b, h, : len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
                seen = torch.zeros(1, k.shape[0], dtype=torch.bool, device="cuda")
                seen[0, (torch.tensor(chosen)[:, None] * bl + torch.arange(bl)).flatten()] = True
                seen[0, n:] = False
            else:
                seen = (torch.arange(k.shape[0], device="cuda") < n)[None]
            O[b, :, h] = _exact_softmax(q, k, v, seen, s["scale"]).view(T, G, d)
    out = {"O": O.view(s["Q"].shape)}
    if op == "qstep":
        out |= {"K": back[0], "V": back[1], "scales": s["scales"].to(F64)}
    if op == "bstep":
        out |= {"idx": idx, "bsum": bsum}
    return out
