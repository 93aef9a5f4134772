"""Plain 64-bit forms of the operators on new tokens and e4m3 caches, one row
at a time from their definitions (test infrastructure only).  CPU float64
throughout; inputs are the tensors a call gets, moved here."""
import math

import torch

F8 = torch.float8_e4m3fn


def cpu(t):
    return None if t is None else t.detach().cpu()


def norm_rope(x, weight, pos, inv_freq, interleaved=False, scale=1.0, eps=1e-6):
    """Rows x [n][H][D] at positions pos [n] -> float64 [n][H][D]."""
    y = cpu(x).double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * cpu(weight).double()
    f = cpu(inv_freq).double()
    h = f.numel()
    ang = cpu(pos).double()[:, None, None] * f
    c, s = torch.cos(ang) * scale, torch.sin(ang) * scale
    first = torch.arange(h) * 2 if interleaved else torch.arange(h)
    second = first + 1 if interleaved else first + h
    out = y.clone()
    out[..., first] = y[..., first] * c - y[..., second] * s
    out[..., second] = y[..., second] * c + y[..., first] * s
    return out


def quantise_row(x):
    """One bf16 row (float64 list) -> (values of its codes float64, scale byte)."""
    x = cpu(x).double()
    if not torch.isfinite(x).all():
        return torch.full_like(x, math.nan), 255
    most = float(x.abs().max())
    e = 16
    while e < 134 and most > 448.0 * 2.0 ** (e - 127):
        e += 1
    y = (x / 2.0 ** (e - 127)).clamp(-448, 448)
    exp = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), exp - 3)
    return torch.round(y / step) * step, e


def cache_row(cache, scale, block, h, at):
    """A cached row as float64 values."""
    r = cache[block, h, at].double()
    return r if scale is None else (r * 2.0 ** (int(scale[block, h, at]) - 127) if int(scale[block, h, at]) != 255
                                    else torch.full_like(r, math.nan))


def keys_of(cache, scale, table, b, lo, hi, h, bs):
    """Rows lo..hi-1 of sequence b, head h, float64 [hi - lo][D]."""
    cache, scale, table = cpu(cache), cpu(scale), cpu(table)
    rows = [cache_row(cache, scale, int(table[b, j // bs]), h, j % bs) for j in range(lo, hi)]
    return torch.stack(rows) if rows else torch.zeros((0, cache.shape[-1]), dtype=torch.float64)


def attend(q, k, v, scale):
    """Softmax attention of one row over the keys it sees: (out, lse, sum w |v|)."""
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, -math.inf, z
    s = (k @ q) * scale
    lse = torch.logsumexp(s, 0)
    w = torch.exp(s - lse)
    return w @ v, float(lse), w @ v.abs()


def chunk_rows(q, k_cache, v_cache, table, prefix_len, q_start, window=0, k_scale=None, v_scale=None, scale=0.0,
               rows=None):
    """{(token, head): (out, lse, sum w|v|)} for the given rows (all if None)."""
    qc, bs = cpu(q).double(), k_cache.shape[2]
    N, Hq, D = q.shape
    G = Hq // k_cache.shape[1]
    s = scale if scale > 0 else 1.0 / math.sqrt(D)
    start, pre = cpu(q_start).tolist(), cpu(prefix_len).tolist()
    k_cache, v_cache, table, k_scale, v_scale = map(cpu, (k_cache, v_cache, table, k_scale, v_scale))
    got, held = {}, {}
    for b in range(len(pre)):
        for t in range(start[b], start[b + 1]):
            for h in range(Hq):
                if rows is not None and (t, h) not in rows:
                    continue
                pos = pre[b] + t - start[b]
                lo = max(0, pos - window + 1) if window > 0 else 0
                key = (b, h // G)
                if key not in held:
                    first = max(0, pre[b] - window + 1) if window > 0 else 0
                    hi = pre[b] + start[b + 1] - start[b]
                    held[key] = (first, keys_of(k_cache, k_scale, table, b, first, hi, h // G, bs),
                                 keys_of(v_cache, v_scale, table, b, first, hi, h // G, bs))
                first, k, v = held[key]
                got[(t, h)] = attend(qc[t, h], k[lo - first:pos + 1 - first], v[lo - first:pos + 1 - first], s)
    return got


def tree_rows(q, k_cache, v_cache, table, prefix_len, k_tree, v_tree, parent, k_scale, v_scale, scale=0.0):
    """(out [B][Hq][T][D], lse, sum w|v|) of verification over an e4m3 cache;
    k_tree None: the prefix alone."""
    B, Hq, T, D = q.shape
    Hkv, bs = k_cache.shape[1], k_cache.shape[2]
    s = scale if scale > 0 else 1.0 / math.sqrt(D)
    out = torch.zeros((B, Hq, T, D), dtype=torch.float64)
    absv, lse = torch.zeros_like(out), torch.zeros((B, Hq, T), dtype=torch.float64)
    qc = cpu(q).double()
    for b in range(B):
        L = int(prefix_len[b])
        for h in range(Hkv):
            k = keys_of(k_cache, k_scale, table, b, 0, L, h, bs)
            v = keys_of(v_cache, v_scale, table, b, 0, L, h, bs)
            for t in range(T):
                kk, vv = k, v
                if k_tree is not None:
                    path, up = [], t
                    while up >= 0:
                        path.append(up)
                        up = int(parent[b, up])
                    kk = torch.cat((k, cpu(k_tree)[b, h, path].double()))
                    vv = torch.cat((v, cpu(v_tree)[b, h, path].double()))
                for g in range(Hq // Hkv):
                    i = h * (Hq // Hkv) + g
                    out[b, i, t], lse[b, i, t], absv[b, i, t] = attend(qc[b, i, t], kk, vv, s)
    return out, lse, absv


# Half a rounding step, relative: the unit every bound below counts in.
BF16 = torch.finfo(torch.bfloat16).eps / 2
E4M3 = torch.finfo(torch.float8_e4m3fn).eps / 2
F32 = torch.finfo(torch.float32).eps / 2


def check_attention(out, lse, ref, ref_lse, absv, scores=32.0, what=""):
    """out against ref, per value: the output's rounding, 2^-8 |ref|; the
    weights, rounded to bf16 before they meet V while their sum is taken over
    the rounded ones, so each weight is off by 2 * 2^-8 at most and the value
    by that times sum w|v|; the scores, fp32 sums of 128 products of size up
    to `scores`, and the exponentials (1e-4 relative), which move a weight by
    less than 2 * (1e-4 + 128 * 2^-24 * scores).  lse: the same score and
    exponential terms, once."""
    out, lse = cpu(out).double(), cpu(lse).double()
    soft = 1e-4 + 128 * F32 * scores
    bound = BF16 * ref.abs() + (2 * BF16 + 2 * soft) * absv * (1 + BF16) + 1e-30
    bad = (out - ref).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float(((out - ref).abs() - bound).max()):.3e}"
    empty = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse), empty), what
    d = (lse - ref_lse).abs()[~empty]
    assert not d.numel() or float(d.max()) <= soft + 4 * F32 * scores, f"{what}: lse off by {float(d.max()):.3e}"
