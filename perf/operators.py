"""Cases of the operators that take tokens into a paged KV cache and read it back.

qk_norm_rope    norm of each query and key head, and its position rotation
append          new K/V rows into a paged cache, bf16 or e4m3 with a power-of-two scale per row;
                with the norm and the rotation in the same pass ("rope": true)
chunk           causal attention of ragged chunks of new tokens over the paged cache that holds them
verify_q8       tree verification over a paged cache held in e4m3

With `own` false, run() computes each operator from its formula in plain torch operations; with
`own` true it makes the calls a user makes of tree_masked_verification_b200.hta.

e4m3 cache rows: row x of D values is stored as codes c and one byte e, x ~ c * 2^(e - 127), where
2^(e - 127) is the smallest power of two with max|x| <= 448 * 2^(e - 127), e clamped to [16, 134].
"""
import math

import torch

own = False

ROPE_BASE = 500000.0


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one sequence in a decode step, heads of 40 over 8, norms on: latency only
        {"name": "rope-token", "op": "qk_norm_rope", "layout": "tokens", "B": 1, "T": 1, "Hq": 40, "Hkv": 8,
         "D": 128, "rot": 128, "interleaved": False, "norm": True, "pos0": 32768},
        # the 68-node draft tree of eight sequences, from projection rows into the verification layout
        {"name": "rope-tree-b8", "op": "qk_norm_rope", "layout": "heads", "B": 8, "T": 68, "Hq": 32, "Hkv": 32,
         "D": 128, "rot": 128, "interleaved": False, "norm": False, "pos0": 16384},
        # a long prompt chunk far into a 256k context: norms, interleaved pairs, half of the head
        {"name": "rope-chunk-16k", "op": "qk_norm_rope", "layout": "tokens", "B": 1, "T": 16384, "Hq": 32,
         "Hkv": 8, "D": 128, "rot": 64, "interleaved": True, "norm": True, "pos0": 245760},
        # one new token of each of 64 sequences into an e4m3 cache: latency and scattered rows
        {"name": "append-q8-tokens", "op": "append", "B": 64, "tmin": 1, "tmax": 1, "pmin": 1000, "pmax": 4000,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 16, "q8": True, "rope": False, "norm": False},
        # ragged prompt chunks, rotated and written to a bf16 cache in one pass
        {"name": "append-rope-ragged", "op": "append", "B": 7, "tmin": 1, "tmax": 1900, "pmin": 0, "pmax": 2500,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 32, "q8": False, "rope": True, "norm": True},
        # a whole batch's prompts of multi-head K/V into an e4m3 cache: bandwidth
        {"name": "append-q8-16k", "op": "append", "B": 4, "tmin": 4096, "tmax": 4096, "pmin": 0, "pmax": 0,
         "Hq": 32, "Hkv": 32, "D": 128, "bs": 64, "q8": True, "rope": False, "norm": False},
        # one decode step of 16 sequences of 4k to 32k keys: the cache is read once
        {"name": "chunk-decode-b16", "op": "chunk", "B": 16, "tmin": 1, "tmax": 1, "pmin": 4096, "pmax": 32767,
         "Hq": 32, "Hkv": 8, "D": 128, "bs": 64, "q8": False, "window": 0},
        # one token of one sequence of 256k keys in e4m3: one long axis, split and joined
        {"name": "chunk-decode-q8-256k", "op": "chunk", "B": 1, "tmin": 1, "tmax": 1, "pmin": 262143,
         "pmax": 262143, "Hq": 32, "Hkv": 8, "D": 128, "bs": 128, "q8": True, "window": 0},
        # ragged chunks and single tokens together, sliding window of 512 (a draft block's own heads of 64)
        {"name": "chunk-window-ragged", "op": "chunk", "B": 9, "tmin": 1, "tmax": 700, "pmin": 0, "pmax": 3000,
         "Hq": 28, "Hkv": 4, "D": 64, "bs": 16, "q8": False, "window": 512},
        # a 4k chunk of a prompt behind 12k keys: compute
        {"name": "chunk-prefill-4k-16k", "op": "chunk", "B": 1, "tmin": 4096, "tmax": 4096, "pmin": 12288,
         "pmax": 12288, "Hq": 32, "Hkv": 8, "D": 128, "bs": 64, "q8": False, "window": 0},
        # the 68-node tree over 32k keys in e4m3, heads of 32 over 8
        {"name": "verify-q8-32k", "op": "verify_q8", "B": 1, "T": 68, "pmin": 32768, "pmax": 32768, "Hq": 32,
         "Hkv": 8, "D": 128, "bs": 64},
        # the same tree for eight sequences of 8k to 16k keys, 32 heads each: the cache's bytes
        {"name": "verify-q8-b8", "op": "verify_q8", "B": 8, "T": 68, "pmin": 8192, "pmax": 16384, "Hq": 32,
         "Hkv": 32, "D": 128, "bs": 32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "append", "chunk", "chunk", "verify_q8"])
    Hq, Hkv = rng.choice([(32, 8), (40, 8), (32, 32), (28, 4), (8, 2), (16, 1), (2, 1)])
    D = rng.choice([64, 128, 128])
    bs = rng.choice([16, 32, 64, 128])
    if op == "qk_norm_rope":
        layout = rng.choice(["tokens", "heads"])
        B = 1 if layout == "tokens" else _log(rng, 1, 16)
        T = _log(rng, 1, 16384 if layout == "tokens" else 256)
        rot = rng.choice([D, D, D // 2, D // 4, D - 2 * rng.randrange(1, D // 2)])
        return {"op": op, "layout": layout, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
                "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.5, "pos0": _log(rng, 1, 1000000)}
    if op == "append":
        q8 = rng.random() < 0.5
        B = _log(rng, 1, 64)
        tmax = _log(rng, 1, max(1, 16384 // B))
        pmax = _log(rng, 1, max(1, 32768 // B))
        return {"op": op, "B": B, "tmin": rng.choice([1, tmax]), "tmax": tmax, "pmin": 0, "pmax": pmax, "Hq": Hq,
                "Hkv": Hkv, "D": D, "bs": bs, "q8": q8, "rope": not q8 and rng.random() < 0.7,
                "norm": rng.random() < 0.5}
    if op == "chunk":
        tmax = rng.choice([1, _log(rng, 1, 4096)])
        B = _log(rng, 1, 16 if tmax > 1 else 32)
        pmax = _log(rng, 1, 131072 // (B if B * tmax > 64 else max(1, B // 8)))
        while B * Hq * tmax * (tmax + pmax) > 32 * 4096 * 16384 // 2:   # no dearer than the largest listed one
            tmax, pmax = max(1, tmax // 2), max(1, pmax // 2)
        return {"op": op, "B": B, "tmin": rng.choice([1, tmax]), "tmax": tmax, "pmin": rng.choice([0, pmax]),
                "pmax": pmax, "Hq": Hq, "Hkv": Hkv, "D": D, "bs": bs, "q8": rng.random() < 0.4,
                "window": rng.choice([0, 0, 0, _log(rng, 1, 2048)])}
    B = _log(rng, 1, 8)
    pmax = _log(rng, 1, 32768 // max(1, B // 2))
    return {"op": op, "B": B, "T": rng.choice([1, 5, 68, rng.randrange(1, 257)]), "pmin": rng.choice([0, pmax]),
            "pmax": pmax, "Hq": Hq, "Hkv": Hkv, "D": D, "bs": bs}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _lens(case):
    """Prefix lengths and chunk lengths, host lists: the case's own, whatever the seed."""
    g = torch.Generator()
    g.manual_seed(11)
    B = case["B"]
    pre = torch.randint(case["pmin"], case["pmax"] + 1, (B,), generator=g).tolist()
    n = torch.randint(case["tmin"], case["tmax"] + 1, (B,), generator=g).tolist() if "tmin" in case else [0] * B
    return pre, n


def _table(case, held, seed):
    """Shuffled blocks for held[b] keys of each sequence; -1 behind a sequence's last block."""
    bs = case["bs"]
    used = [-(-h // bs) for h in held]
    n, most = sum(used) + 2, max(1, max(used))
    g = torch.Generator()
    g.manual_seed(seed + 2)
    perm = torch.randperm(n, generator=g).to(torch.int32)
    table = torch.full((case["B"], most), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    return table.cuda(), n, most * bs


def _power(e):
    """2^(e - 127) in fp32, exactly, for e from 1 to 254."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _quantise(x):
    """bf16 rows [..., D] -> (codes e4m3 [..., D], scale bytes [...])."""
    amax = x.abs().amax(-1).float()
    mant, ex = torch.frexp(amax)                           # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, ex - 9 + (mant > 0.875).to(ex.dtype) + 127, 16).clamp(16, 134)
    y = (x.float() * _power(254 - e)[..., None]).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn), e.to(torch.uint8)


def _inv_freq(rot):
    return (ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).to(torch.float32).cuda()


def prepare(case, seed):
    op, Hq, Hkv, D = case["op"], case["Hq"], case["Hkv"], case["D"]
    g = _gen(seed)
    s = {"case": case}
    if op in ("qk_norm_rope", "append") and (op == "qk_norm_rope" or case["rope"]):
        s["inv_freq"] = _inv_freq(case.get("rot", D))
        s["rope_scale"] = 1.0
        s["q_weight"] = (1 + 0.2 * _randn(g, D)) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * _randn(g, D)) if case["norm"] else None
    if op == "qk_norm_rope":
        B, T = case["B"], case["T"]
        qkv = _randn(g, B * T, (Hq + 2 * Hkv) * D)        # the projection's rows
        q, k = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D]
        if case["layout"] == "tokens":
            s["q"], s["k"] = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D))
            s["positions"] = (case["pos0"] + torch.arange(T)).to(torch.int32).cuda()
        else:
            s["q"] = q.unflatten(1, (Hq, D)).unflatten(0, (B, T)).transpose(1, 2)
            s["k"] = k.unflatten(1, (Hkv, D)).unflatten(0, (B, T)).transpose(1, 2)
            hg = torch.Generator()
            hg.manual_seed(seed + 3)
            base = torch.randint(0, case["pos0"] + 1, (B, 1), generator=hg)
            s["positions"] = (base + torch.randint(0, 6, (B, T), generator=hg)).to(torch.int32).cuda()
        return s

    pre, n = _lens(case)
    s["prefix_len"] = torch.tensor(pre, dtype=torch.int32).cuda()
    held = [p + m for p, m in zip(pre, n)]
    s["table"], blocks, s["L_cap"] = _table(case, held, seed)
    shape = (blocks, Hkv, case["bs"], D)
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _randn(g, *shape), _randn(g, *shape), None, None
    if case.get("q8", True):
        s["k_cache"], s["k_scale"] = _quantise(s["k_cache"])
        s["v_cache"], s["v_scale"] = _quantise(s["v_cache"])
    s["keys"] = max(1, max(held))
    if op == "verify_q8":
        B, T = case["B"], case["T"]
        s["q"], s["k_tree"], s["v_tree"] = _randn(g, B, Hq, T, D), _randn(g, B, Hkv, T, D), _randn(g, B, Hkv, T, D)
        hg = torch.Generator()
        hg.manual_seed(seed + 3)
        parent = torch.full((B, T), -1, dtype=torch.int32)
        for i in range(4, T):                               # four roots, then a parent among the last 20 nodes
            parent[:, i] = torch.randint(max(0, i - 20), i, (B,), generator=hg).to(torch.int32)
        s["parent"] = parent.cuda()
        return s
    s["q_start"] = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32).cuda()
    s["longest"] = max(n)
    N = sum(n)
    if op == "append":
        qkv = _randn(g, N, (Hq + 2 * Hkv) * D)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    else:
        s["q"] = _randn(g, N, Hq, D)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _plain_rows(x, weight, cos, sin, rot, interleaved):
    """Norm (where there is a weight) and rotation of rows [..., D] in 32 bits; cos/sin [..., rot/2]."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1).to(torch.bfloat16)


def _plain_angles(positions, inv_freq, scale):
    """cos and sin in 64 bits, for far positions."""
    a = positions.double()[..., None] * inv_freq.double()
    return (a.cos() * scale).float(), (a.sin() * scale).float()


def _plain_keys(cache, scale, table, keys):
    """The cached rows of each sequence in key order, fp32 [B, Hkv, keys, D]."""
    at = table.clamp(min=0).long()
    x = cache[at].float()
    if scale is not None:
        x = x * _power(scale[at])[..., None]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :keys]


def _plain_tokens(s):
    """Sequence and place in its chunk of each new token."""
    N, start = s["q"].shape[0], s["q_start"].long()
    i = torch.arange(N, device="cuda")
    seq = torch.searchsorted(start[1:], i, right=True)
    return seq, i - start[seq]


def _plain_softmax(scores, keep):
    """exp(scores - max), its sum and the lse over the last axis, where `keep`."""
    scores = scores.masked_fill(~keep, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    return p, total, (m + total.log()).squeeze(-1)


def _plain_chunk(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    seq, t = _plain_tokens(s)
    q = torch.zeros((B, s["longest"], Hq, D), device="cuda")
    q[seq, t] = s["q"].float()
    q = q.transpose(1, 2).unflatten(1, (Hkv, Hq // Hkv))              # [B, Hkv, G, t, D]
    k = _plain_keys(s["k_cache"], s["k_scale"], s["table"], s["keys"])
    v = _plain_keys(s["v_cache"], s["v_scale"], s["table"], s["keys"])
    j = torch.arange(s["keys"], device="cuda")
    pos = s["prefix_len"][:, None, None] + torch.arange(s["longest"], device="cuda")[:, None]
    keep = j <= pos                                                   # [B, t, key]
    if case["window"]:
        keep = keep & (j > pos - case["window"])
    scores = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, q.shape[2:4]) / math.sqrt(D)
    p, total, lse = _plain_softmax(scores, keep[:, None, None])
    out = (p.flatten(2, 3) @ v).unflatten(2, q.shape[2:4]) / total
    out = out.flatten(1, 2).transpose(1, 2)[seq, t]
    return out.to(torch.bfloat16), lse.flatten(1, 2).transpose(1, 2)[seq, t]


def _plain_verify(s):
    case = s["case"]
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    q = s["q"].float().unflatten(1, (Hkv, Hq // Hkv))                 # [B, Hkv, G, T, D]
    k = torch.cat((_plain_keys(s["k_cache"], s["k_scale"], s["table"], s["keys"]), s["k_tree"].float()), 2)
    v = torch.cat((_plain_keys(s["v_cache"], s["v_scale"], s["table"], s["keys"]), s["v_tree"].float()), 2)
    step = (s["parent"][..., None] == torch.arange(T, device="cuda")).double()
    eye = torch.eye(T, dtype=torch.float64, device="cuda")
    above = torch.linalg.matrix_power((eye + step) / 2, 256) > 0      # node or ancestor of it, up to 256 up
    before = (torch.arange(s["keys"], device="cuda") < s["prefix_len"][:, None])[:, None].expand(-1, T, -1)
    keep = torch.cat((before, above), -1)                             # [B, T, key]
    scores = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, q.shape[2:4]) / math.sqrt(D)
    p, total, lse = _plain_softmax(scores, keep[:, None, None])
    out = (p.flatten(2, 3) @ v).unflatten(2, q.shape[2:4]) / total
    return out.flatten(1, 2).to(torch.bfloat16), lse.flatten(1, 2)


def _plain_append(s):
    case = s["case"]
    seq, t = _plain_tokens(s)
    pos = s["prefix_len"][seq] + t
    block = s["table"][seq, pos // case["bs"]].long()
    at = pos % case["bs"]
    k, v, q = s["k"], s["v"], None
    if case["rope"]:
        cos, sin = _plain_angles(pos[:, None], s["inv_freq"], s["rope_scale"])
        q = _plain_rows(s["q"], s["q_weight"], cos, sin, case["D"], False)
        k = _plain_rows(k, s["k_weight"], cos, sin, case["D"], False)
    if not case["q8"]:
        s["k_cache"][block, :, at] = k
        s["v_cache"][block, :, at] = v
        return q, s["k_cache"], s["v_cache"]
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    s["k_cache"].view(torch.uint8)[block, :, at] = kc.view(torch.uint8)
    s["v_cache"].view(torch.uint8)[block, :, at] = vc.view(torch.uint8)
    s["k_scale"][block, :, at] = ks
    s["v_scale"][block, :, at] = vs
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain(s):
    case = s["case"]
    if case["op"] == "qk_norm_rope":
        p = s["positions"]
        cos, sin = _plain_angles(p[:, None] if p.dim() == 1 else p[:, None, :], s["inv_freq"], s["rope_scale"])
        return tuple(_plain_rows(s[x], s[x + "_weight"], cos, sin, case["rot"], case["interleaved"]) for x in "qk")
    return {"append": _plain_append, "chunk": _plain_chunk, "verify_q8": _plain_verify}[case["op"]](s)


# ------------------------------------------------------------------------------------ the framework's calls
def _own(s):
    from tree_masked_verification_b200 import hta
    case = s["case"]
    if case["op"] == "qk_norm_rope":
        return hta.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                                k_weight=s["k_weight"], eps=1e-6, interleaved=case["interleaved"],
                                rope_scale=s["rope_scale"])
    cache = {"L_cap": s["L_cap"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if case["op"] == "append":
        if "ws" not in s:
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")     # the status word
        if case["rope"]:
            q = hta.rope_append_paged(s["q"], s["k"], s["v"], s["inv_freq"], s["k_cache"], s["v_cache"], s["table"],
                                      s["prefix_len"], s["q_start"], q_weight=s["q_weight"],
                                      k_weight=s["k_weight"], eps=1e-6, rope_scale=s["rope_scale"],
                                      workspace=s["ws"], **cache)
            return q, s["k_cache"], s["v_cache"]
        hta.append_paged(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], s["q_start"],
                         workspace=s["ws"], **cache)
        if case["q8"]:
            return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        return None, s["k_cache"], s["v_cache"]
    if case["op"] == "chunk":
        if "ws" not in s:
            s["ws"] = hta.new_chunk_workspace(s["q"], s["k_cache"], case["B"], L_cap=s["L_cap"])
        return hta.chunk_attention_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"],
                                         s["q_start"], window=case["window"], workspace=s["ws"], **cache)
    if "ws" not in s:
        s["ws"] = hta.new_q8_workspace(hta.Dims(case["B"], case["Hq"], case["Hkv"], case["D"], case["T"], s["L_cap"], 0.0))
    return hta.verify_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["prefix_len"], s["k_tree"],
                            s["v_tree"], s["parent"], workspace=s["ws"], **cache)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ floors
def work(case):
    op, Hq, Hkv, D = case["op"], case["Hq"], case["Hkv"], case["D"]
    if op == "qk_norm_rope":
        n = case["B"] * case["T"]
        return {"bytes": n * (4 * (Hq + Hkv) * D + 4), "flops": n * (Hq + Hkv) * (3 * case["rot"] + 4 * D * case["norm"])}
    row = (D + 1 if case.get("q8", True) else 2 * D) * 2 * Hkv           # one key's K and V in the cache
    pre, new = _lens(case)
    if op == "append":
        n = sum(new)
        q = 4 * Hq * D if case["rope"] else 0
        return {"bytes": n * (4 * Hkv * D + row + q), "flops": n * (3 * (Hq + Hkv) * D if case["rope"] else 2 * Hkv * D)}
    if op == "chunk":
        w = case["window"] or 1 << 40
        read = sum(min(p, w - 1) + m for p, m in zip(pre, new))
        seen = sum(min(p + t + 1, w) for p, m in zip(pre, new) for t in range(m))
        return {"bytes": read * row + sum(new) * Hq * (4 * D + 4), "flops": 4 * Hq * D * seen}
    T, B = case["T"], case["B"]
    return {"bytes": sum(pre) * row + B * T * (4 * Hq * D + 4 * Hq + 4 * Hkv * D + 4),
            "flops": 4 * T * Hq * D * (sum(pre) + B * min(T, 5))}


# ------------------------------------------------------------------------------------ 64 bits
def _exact_rotate(x, weight, pos, inv_freq, rot, interleaved):
    """Rows [n, H, D] at positions [n]: each pair as a complex number times e^(i * position * frequency)."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * weight.double()
    w = inv_freq.double()
    turn = torch.polar(torch.ones_like(w).expand(len(pos), -1), pos.double()[:, None] * w)[:, None]
    y = x.clone()
    if interleaved:
        first, second = list(range(0, rot, 2)), list(range(1, rot, 2))
    else:
        first, second = list(range(rot // 2)), list(range(rot // 2, rot))
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_powers():
    return torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device="cuda")


def _exact_codes(x):
    """Values of the e4m3 codes of rows x: three bits behind the leading one, steps of 2^-9 below 2^-6."""
    most = x.abs().amax(-1, keepdim=True)
    powers = _exact_powers()
    unit = powers[torch.searchsorted(powers, (most / 448).contiguous()).clamp(16, 134)]
    y = (x / unit).clamp(-448, 448)
    step = powers[torch.searchsorted(powers, y.abs().clamp(min=2.0 ** -6), right=True) - 1] / 8
    return torch.round(y / step) * step


def _exact_cached(cache, scale, table, b, n, bs, h):
    """Keys 0..n-1 of sequence b, head h."""
    blocks = table[b, :max(1, -(-n // bs))].long()
    x = cache[blocks, h].double()
    if scale is not None:
        x = x * _exact_powers()[scale[blocks, h].long()][..., None]
    return x.reshape(-1, x.shape[-1])[:n]


def _exact_attend(q, k, v, keep):
    s = (q @ k.T) / math.sqrt(q.shape[-1])
    s = torch.where(keep, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op, B, Hq, Hkv, D = case["op"], case["B"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    if op == "qk_norm_rope":
        got = []
        for x in "qk":
            rows = s[x] if s[x].dim() == 3 else s[x].transpose(1, 2).reshape(B * case["T"], -1, D)
            y = _exact_rotate(rows, s[x + "_weight"], s["positions"].reshape(-1), s["inv_freq"], case["rot"],
                              case["interleaved"])
            got.append(y if s[x].dim() == 3 else y.unflatten(0, (B, case["T"])).transpose(1, 2))
        return tuple(got)
    pre = s["prefix_len"].tolist()
    if op == "append":
        start = s["q_start"].tolist()
        kc, vc, qs = s["k_cache"].double(), s["v_cache"].double(), []
        for b in range(B):
            at = slice(start[b], start[b + 1])
            pos = pre[b] + torch.arange(start[b + 1] - start[b], device="cuda")
            k = s["k"][at].double()
            if case["rope"]:
                k = _exact_rotate(k, s["k_weight"], pos, s["inv_freq"], D, False)
                qs.append(_exact_rotate(s["q"][at], s["q_weight"], pos, s["inv_freq"], D, False))
            block = s["table"][b][pos // case["bs"]].long()
            v = s["v"][at].double()
            kc[block, :, pos % case["bs"]] = _exact_codes(k) if case["q8"] else k
            vc[block, :, pos % case["bs"]] = _exact_codes(v) if case["q8"] else v
        if case["q8"]:
            return kc, vc, None, None
        return torch.cat(qs) if qs else None, kc, vc
    bs = case["bs"]
    if op == "chunk":
        start = s["q_start"].tolist()
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        for b in range(B):
            n = start[b + 1] - start[b]
            pos = pre[b] + torch.arange(n, device="cuda")[:, None]
            j = torch.arange(pre[b] + n, device="cuda")
            keep = (j <= pos) & ((pos - j < case["window"]) if case["window"] else (j >= 0))
            for h in range(Hkv):
                k = _exact_cached(s["k_cache"], s["k_scale"], s["table"], b, pre[b] + n, bs, h)
                v = _exact_cached(s["v_cache"], s["v_scale"], s["table"], b, pre[b] + n, bs, h)
                for i in range(h * G, h * G + G):
                    at = slice(start[b], start[b + 1])
                    out[at, i], lse[at, i] = _exact_attend(s["q"][at, i].double(), k, v, keep)
        return out, lse
    T = case["T"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    for b, parent in enumerate(s["parent"].tolist()):
        tree = torch.zeros((T, T), dtype=torch.bool)
        for i in range(T):
            up = i
            while up >= 0:
                tree[i, up] = True
                up = parent[up]
        keep = torch.cat((torch.ones((T, pre[b]), dtype=torch.bool), tree), 1).cuda()
        for h in range(Hkv):
            k = _exact_cached(s["k_cache"], s["k_scale"], s["table"], b, pre[b], bs, h)
            v = _exact_cached(s["v_cache"], s["v_scale"], s["table"], b, pre[b], bs, h)
            k, v = torch.cat((k, s["k_tree"][b, h].double())), torch.cat((v, s["v_tree"][b, h].double()))
            for i in range(h * G, h * G + G):
                out[b, i], lse[b, i] = _exact_attend(s["q"][b, i].double(), k, v, keep)
    return out, lse
