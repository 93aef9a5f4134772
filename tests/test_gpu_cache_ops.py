"""Norm and rotation, append, chunk attention and the e4m3 cache against
plain 64-bit forms (needs a B200)."""
import math

import pytest
import torch

from tests import cache_plain as P
from tree_masked_verification_b200 import hta

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()


def freqs(rot, base=500000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def status():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def check_rows(got, x, weight, pos, inv, interleaved, scale=1.0, eps=1e-6):
    ref = P.norm_rope(x, weight, pos, inv, interleaved, scale, eps)
    got = P.cpu(got).double()
    # one rounding to bf16; before it a few dozen fp32 operations on values
    # of the row's size (the norm's sum of D squares among them)
    size = ref.abs().amax(-1, keepdim=True)
    bound = P.BF16 * ref.abs() + 64 * P.F32 * size * 2 + 1e-38
    assert ((got - ref).abs() <= bound).all(), float(((got - ref).abs() - bound).max())


# ------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,rot,interleaved", [
    (128, 128, False), (128, 128, True), (128, 64, False), (128, 64, True), (128, 2, False), (128, 2, True),
    (128, 126, False), (128, 122, True), (64, 64, False), (64, 64, True), (64, 18, False), (64, 34, True)])
def test_rope_tokens(D, rot, interleaved, norm):
    N, Hq, Hkv = 37, 5, 3
    qkv = randn(N, (Hq + 2 * Hkv) * D, seed=D + rot)
    q, k = qkv[:, :Hq * D].unflatten(1, (Hq, D)), qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    pos = torch.tensor([0, 1, 2, 1000003, 262143] + [7 * i * i for i in range(N - 5)], dtype=torch.int32).cuda()
    inv = freqs(rot)
    qw, kw = (randn(D, seed=1), randn(D, seed=2)) if norm else (None, None)
    keep = qkv.clone()
    qo, ko = hta.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, interleaved=interleaved, rope_scale=1.25)
    check_rows(qo, q, qw, pos, inv, interleaved, 1.25)
    check_rows(ko, k, kw, pos, inv, interleaved, 1.25)
    assert torch.equal(qkv, keep)
    # in place, on the slices of the projection's rows
    hta.qk_norm_rope(q, k, pos, inv, q_weight=qw, k_weight=kw, interleaved=interleaved, rope_scale=1.25, q_out=q,
                     k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[:, (Hq + Hkv) * D:], keep[:, (Hq + Hkv) * D:])


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 68, 28, 4), (2, 9, 40, 8), (1, 700, 2, 1)])
def test_rope_heads_layout(B, T, Hq, Hkv):
    D = 128
    q, k = randn(B, T, Hq, D, seed=B + T).transpose(1, 2), randn(B, Hkv, T, D, seed=T)
    pos = torch.randint(0, 5000, (B, T), generator=torch.Generator().manual_seed(T), dtype=torch.int32).cuda()
    inv = freqs(D)
    qo, ko = hta.qk_norm_rope(q, k, pos, inv)
    assert qo.is_contiguous() and qo.shape == q.shape
    for got, x in ((qo, q), (ko, k)):
        check_rows(got.transpose(1, 2).flatten(0, 1), x.transpose(1, 2).flatten(0, 1), None, pos.flatten(), inv, False)


def test_rope_nothing_and_one_sided_weights():
    D, inv = 64, freqs(64)
    qo, ko = hta.qk_norm_rope(randn(0, 4, D), randn(0, 2, D), torch.empty(0, dtype=torch.int32, device="cuda"), inv)
    assert qo.shape == (0, 4, D) and ko.shape == (0, 2, D)
    q, k, w = randn(6, 4, D, seed=3), randn(6, 2, D, seed=4), randn(D, seed=5)
    q[2] = 0                                                  # eps alone under the root
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    qo, ko = hta.qk_norm_rope(q, k, pos, inv, q_weight=w, eps=1e-5)
    check_rows(qo, q, w, pos, inv, False, eps=1e-5)
    check_rows(ko, k, None, pos, inv, False)


# --------------------------------------------------------------------- caches
class Case:
    """Ragged chunks of B sequences over a paged cache with shuffled blocks;
    table entries past a sequence's blocks are out of range, the blocks'
    unused rows hold NaN."""

    def __init__(self, pre, new, Hq, Hkv, D, bs, q8=False, seed=0, pad=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.pre, self.new, self.bs, self.D, self.Hq, self.Hkv = pre, new, bs, D, Hq, Hkv
        held = [p + n for p, n in zip(pre, new)]
        used = [-(-h // bs) for h in held]
        self.L_cap = max(1, max(held))
        most = max(1, max(used))
        perm = torch.randperm(sum(used) + 3, generator=g).int()
        table = torch.full((len(pre), most + 1), -7, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = perm[at:at + u]
            at += u
        self.blocks = len(perm)
        shape = (self.blocks, Hkv, bs, D)
        kc, vc = (torch.full(shape, math.nan, dtype=torch.bfloat16) for _ in range(2))
        for b, h in enumerate(held):
            for j0 in range(0, h, bs):
                n = min(bs, h - j0)
                blk = int(table[b, j0 // bs])
                kc[blk, :, :n] = torch.randn((Hkv, n, D), generator=g).to(torch.bfloat16) * spread
                vc[blk, :, :n] = torch.randn((Hkv, n, D), generator=g).to(torch.bfloat16)
        self.ks = self.vs = None
        if q8:
            (kc, self.ks), (vc, self.vs) = self.quantise(kc), self.quantise(vc)
            self.ks, self.vs = self.ks.cuda(), self.vs.cuda()
        self.kc, self.vc, self.table = kc.cuda(), vc.cuda(), table.cuda()
        start = [sum(new[:b]) for b in range(len(new) + 1)]
        self.q_start = torch.tensor(start, dtype=torch.int32).cuda()
        self.prefix_len = torch.tensor(pre, dtype=torch.int32).cuda()
        self.N = start[-1] + pad
        self.q = torch.randn((self.N, Hq, D), generator=g).to(torch.bfloat16).cuda()

    @staticmethod
    def quantise(x):
        """The stored form of bf16 rows: NaN rows as e = 255 and NaN codes."""
        amax = x.float().abs().amax(-1)
        bad = ~torch.isfinite(amax)
        a = torch.where(bad, torch.ones_like(amax), amax)
        mant, ex = torch.frexp(a)
        e = torch.where(a > 0, ex - 9 + (mant > 0.875).to(ex.dtype) + 127, 16).clamp(16, 134)
        y = (torch.where(bad[..., None], 0.0, x.float()) * torch.pow(2.0, (127 - e).double()).float()[..., None])
        c = y.clamp(-448, 448).to(P.F8).view(torch.uint8)
        c[bad] = 0x7f
        e[bad] = 255
        return c.view(P.F8), e.to(torch.uint8)

    def paged(self):
        return {"L_cap": self.L_cap, "k_scale": self.ks, "v_scale": self.vs}

    def attend(self, window=0, scale=0.0, **kw):
        ws = hta.new_chunk_workspace(self.q, self.kc, len(self.pre), L_cap=self.L_cap)
        out, lse = hta.chunk_attention_paged(self.q, self.kc, self.vc, self.table, self.prefix_len, self.q_start,
                                             window=window, scale=scale, workspace=ws, **self.paged(), **kw)
        return out, lse, hta.get_status(ws)

    def check(self, window=0, scale=0.0, rows=None):
        out, lse, code = self.attend(window, scale)
        assert code == hta.OK
        ref = P.chunk_rows(self.q, self.kc, self.vc, self.table, self.prefix_len, self.q_start, window, self.ks,
                           self.vs, scale, rows)
        at = list(ref)
        t, h = [x[0] for x in at], [x[1] for x in at]
        P.check_attention(out[t, h], lse[t, h], torch.stack([ref[x][0] for x in at]),
                          torch.tensor([ref[x][1] for x in at], dtype=torch.float64),
                          torch.stack([ref[x][2] for x in at]))


def codes(cache, scale):
    return cache.view(torch.uint8), scale


@pytest.mark.parametrize("pre,new,Hq,Hkv,D,bs,pad", [
    ([0], [1], 1, 1, 64, 16, 0), ([5, 0, 130, 17], [3, 0, 20, 1], 8, 2, 128, 16, 3),
    ([0, 0, 64], [64, 0, 100], 28, 4, 64, 32, 0), ([31] * 40, [1] * 40, 4, 4, 128, 64, 1),
    ([100, 1], [129, 127], 40, 8, 128, 128, 0)])
@pytest.mark.parametrize("q8", [False, True])
def test_append(pre, new, Hq, Hkv, D, bs, pad, q8):
    c = Case(pre, new, Hq, Hkv, D, bs, q8, seed=len(pre) + D, pad=pad)
    qkv = randn(c.N, (Hq + 2 * Hkv) * D, seed=5, scale=3.0)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    v = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    if c.N > 2:
        k[0, 0] = 0                                          # a zero row: the least scale
        v[1, -1, 0] = math.inf                               # a row that cannot be held
        k[2, 0] = torch.tensor([2.0 ** -126] * D)            # below the least scale's codes
        v[2, 0, 3] = 6e4                                     # above the largest scale's range
    want_k, want_v = c.kc.clone(), c.vc.clone()
    want_ks, want_vs = (c.ks.clone(), c.vs.clone()) if q8 else (None, None)
    ws = status()
    hta.append_paged(k, v, c.kc, c.vc, c.table, c.prefix_len, c.q_start, workspace=ws, **c.paged())
    assert hta.get_status(ws) == hta.OK
    start = c.q_start.tolist()
    for b in range(len(pre)):
        for t in range(start[b], start[b + 1]):
            pos = pre[b] + t - start[b]
            blk, at = int(c.table[b, pos // bs]), pos % bs
            if q8:
                for src, code, sc in ((k, want_k, want_ks), (v, want_v, want_vs)):
                    for h in range(Hkv):
                        val, e = P.quantise_row(src[t, h])
                        code[blk, h, at] = val.float().to(P.F8).cuda()
                        sc[blk, h, at] = e
            else:
                want_k[blk, :, at], want_v[blk, :, at] = k[t], v[t]
    if q8:
        assert torch.equal(c.ks, want_ks) and torch.equal(c.vs, want_vs)
    for got, want in ((c.kc, want_k), (c.vc, want_v)):       # the whole cache, untouched rows too
        a, b_ = got.view(torch.uint8), want.view(torch.uint8)
        if q8:                                               # NaN codes of either sign, and -0
            a, b_ = (torch.where((x & 0x7f) == 0x7f, 0x7f, x) for x in (a, b_))
        assert torch.equal(a, b_)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("norm,interleaved,rot,D", [(True, False, 128, 128), (False, True, 64, 128),
                                                    (True, False, 32, 64)])
def test_rope_append(q8, norm, interleaved, rot, D):
    Hq, Hkv, bs = 12, 4, 32
    c = Case([40, 0, 7, 1000], [3, 33, 0, 64], Hq, Hkv, D, bs, q8, seed=9, pad=2)
    k, v = randn(c.N, Hkv, D, seed=1), randn(c.N, Hkv, D, seed=2)
    qw, kw = (randn(D, seed=1), randn(D, seed=2)) if norm else (None, None)
    inv, ws = freqs(rot), status()
    q_out = torch.full_like(c.q, 9.0)
    got = hta.rope_append_paged(c.q, k, v, inv, c.kc, c.vc, c.table, c.prefix_len, c.q_start, q_weight=qw,
                                k_weight=kw, interleaved=interleaved, q_out=q_out, workspace=ws, **c.paged())
    assert hta.get_status(ws) == hta.OK and got is q_out
    real = int(c.q_start[-1])
    assert (q_out[real:] == 9.0).all()                       # padding rows stay
    pos = torch.cat([c.pre[b] + torch.arange(n) for b, n in enumerate(c.new)])
    check_rows(q_out[:real], c.q[:real], qw, pos, inv, interleaved)
    ref = P.norm_rope(k[:real], kw, pos, inv, interleaved)
    # the same rows from the two calls in turn
    _, k2 = hta.qk_norm_rope(c.q[:real], k[:real], pos.int().cuda(), inv, q_weight=qw, k_weight=kw,
                             interleaved=interleaved)
    d = Case([40, 0, 7, 1000], [3, 33, 0, 64], Hq, Hkv, D, bs, q8, seed=9)
    hta.append_paged(k2, v[:real], d.kc, d.vc, d.table, d.prefix_len, d.q_start, **d.paged())
    assert torch.equal(c.kc.view(torch.uint8), d.kc.view(torch.uint8))
    assert torch.equal(c.vc.view(torch.uint8), d.vc.view(torch.uint8))
    if q8:
        assert torch.equal(c.ks, d.ks) and torch.equal(c.vs, d.vs)
    kc, ks, table = P.cpu(c.kc), P.cpu(c.ks), P.cpu(c.table)
    i = 0
    for b, n in enumerate(c.new):
        for t in range(n):
            p = c.pre[b] + t
            for h in range(Hkv):
                row = P.cache_row(kc, ks, int(table[b, p // bs]), h, p % bs)
                size = float(ref[i, h].abs().max())
                bound = P.BF16 * ref[i, h].abs() + 128 * P.F32 * size
                if q8:   # a code's rounding: half a step, at least half the least step of the row's scale
                    bound = bound + P.E4M3 * 1.01 * ref[i, h].abs() + size / 224 * 2.0 ** -10
                assert ((row - ref[i, h]).abs() <= bound).all()
            i += 1


def test_append_reports_and_leaves_bad_sequences():
    for case, want in (("len", hta.ERR_PREFIX_LEN_RANGE), ("negative", hta.ERR_PREFIX_LEN_RANGE),
                       ("block", hta.ERR_BAD_BLOCK), ("order", hta.ERR_BAD_RANGES), ("over", hta.ERR_BAD_RANGES)):
        c = Case([10, 20, 5], [4, 3, 2], 4, 2, 64, 16, seed=3)
        k, v, ws = randn(c.N, 2, 64, seed=1), randn(c.N, 2, 64, seed=2), status()
        before = c.kc.clone()
        if case == "len":
            c.prefix_len[1] = c.L_cap - 2
        elif case == "negative":
            c.prefix_len[1] = -1
        elif case == "block":
            c.table[1, 1] = c.blocks
        elif case == "order":
            c.q_start[1] = 8
        else:
            c.q_start[3] = c.N + 1
        q_out = torch.zeros_like(c.q)
        hta.rope_append_paged(c.q, k, v, freqs(64), c.kc, c.vc, c.table, c.prefix_len, c.q_start, q_out=q_out,
                              workspace=ws, **c.paged())
        assert hta.get_status(ws) == want, case
        if case in ("len", "negative", "block"):
            changed = (c.kc.view(torch.uint8) != before.view(torch.uint8)).flatten(1).any(1)
            blk = [int(c.table[1, i]) for i in range(2)]
            assert not any(bool(changed[i]) for i in blk if i < c.blocks), case
            assert torch.isnan(q_out[4:7]).all() and torch.isfinite(q_out[:4]).all() and torch.isfinite(q_out[7:]).all()


# ------------------------------------------------------------ chunk attention
SHAPES = [
    ([0], [1], 1, 1, 64, 16), ([0], [3], 4, 1, 128, 128), ([127], [1], 4, 4, 128, 16), ([128], [1], 8, 2, 64, 32),
    ([0, 300, 5], [130, 1, 17], 8, 2, 128, 16), ([255, 0, 64, 1], [2, 0, 65, 128], 28, 4, 64, 64),
    ([1000], [40], 16, 1, 128, 64), ([3, 700, 129], [1, 1, 1], 40, 8, 128, 16), ([90], [300], 2, 1, 128, 128),
    ([0, 2], [0, 1], 2, 2, 64, 16), ([513, 40, 7, 260], [1, 257, 5, 31], 5, 5, 128, 32),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("window", [0, 1, 100, 512])
@pytest.mark.parametrize("pre,new,Hq,Hkv,D,bs", SHAPES)
def test_chunk_attention(pre, new, Hq, Hkv, D, bs, window, q8):
    Case(pre, new, Hq, Hkv, D, bs, q8, seed=sum(pre) + D + window).check(window)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("pre,new,Hq,Hkv,D,bs", [
    ([9000], [1], 8, 2, 128, 64), ([5000, 20, 8191], [1, 1, 2], 4, 1, 64, 32), ([3000], [500], 8, 2, 128, 128)])
def test_chunk_attention_long(pre, new, Hq, Hkv, D, bs, q8):
    """Long axes, split over the GPU and joined; a few rows of each call."""
    c = Case(pre, new, Hq, Hkv, D, bs, q8, seed=1)
    rows = {(t, h) for t in {0, 1, c.N // 2, c.N - 1} for h in (0, Hq - 1)}
    c.check(0, rows=rows)
    c.check(700, rows=rows)


@pytest.mark.parametrize("q8", [False, True])
def test_chunk_attention_peaked_scores_and_scale(q8):
    """Scores of hundreds (one key takes the row) and a scale of the caller's."""
    c = Case([300, 10], [40, 1], 8, 2, 128, 16, q8, seed=4, spread=8.0)
    out, lse, code = c.attend(scale=0.02)
    c.check(scale=0.02)
    c.q *= 4
    ref = P.chunk_rows(c.q, c.kc, c.vc, c.table, c.prefix_len, c.q_start, 0, c.ks, c.vs)
    out, lse, code = c.attend()
    at = list(ref)
    t, h = [x[0] for x in at], [x[1] for x in at]
    P.check_attention(out[t, h], lse[t, h], torch.stack([ref[x][0] for x in at]),
                      torch.tensor([ref[x][1] for x in at], dtype=torch.float64),
                      torch.stack([ref[x][2] for x in at]), scores=400.0)


def test_chunk_attention_leaves_padding_and_takes_strided_queries():
    c = Case([50, 3], [30, 2], 8, 2, 128, 32, seed=2, pad=5)
    wide = torch.zeros((c.N, 12, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = c.q
    out = torch.full_like(c.q, 5.0)
    lse = torch.full(c.q.shape[:2], 5.0, device="cuda")
    c.attend(out=out, lse=lse)
    assert (out[32:] == 5.0).all() and (lse[32:] == 5.0).all()
    c.q = wide[:, :8]
    out2, lse2, _ = c.attend()
    assert torch.equal(out2[:32], out[:32]) and torch.equal(lse2[:32], lse[:32])


def test_chunk_attention_reports():
    for case, want in (("len", hta.ERR_PREFIX_LEN_RANGE), ("block", hta.ERR_BAD_BLOCK), ("order", hta.ERR_BAD_RANGES)):
        c = Case([40, 20, 5], [4, 3, 2], 4, 2, 64, 16, seed=3)
        good, _, _ = c.attend()
        if case == "len":
            c.prefix_len[1] = c.L_cap
        elif case == "block":
            c.table[1, 0] = c.blocks
        else:
            c.q_start[1] = 8
        out, lse, code = c.attend()
        assert code == want, case
        if case == "len":
            assert torch.isnan(out[4:7].float()).all() and torch.isnan(lse[4:7]).all()
        if case != "order":
            assert torch.equal(out[:4], good[:4]) and torch.equal(out[7:], good[7:])


# ----------------------------------------------------- trees over e4m3 caches
@pytest.mark.parametrize("pre,Hq,Hkv,T,D,bs", [
    ([0], 1, 1, 1, 64, 16), ([300], 8, 2, 68, 128, 64), ([0, 129, 1], 4, 4, 5, 128, 16), ([700, 3], 28, 4, 33, 64, 32),
    ([40], 2, 1, 256, 128, 128), ([513], 16, 1, 17, 128, 16)])
def test_verify_and_prefix_attention_q8(pre, Hq, Hkv, T, D, bs):
    c = Case(pre, [0] * len(pre), Hq, Hkv, D, bs, True, seed=T + D)
    B = len(pre)
    q, kt, vt = randn(B, Hq, T, D, seed=1), randn(B, Hkv, T, D, seed=2), randn(B, Hkv, T, D, seed=3)
    g = torch.Generator().manual_seed(T)
    parent = torch.tensor([[int(torch.randint(max(-1, i - 9), i, (1,), generator=g)) for i in range(T)]
                           for _ in range(B)], dtype=torch.int32).cuda()
    ws = hta.new_q8_workspace(hta.Dims(B, Hq, Hkv, D, T, c.L_cap, 0.0))
    out, lse = hta.verify_paged(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, workspace=ws, **c.paged())
    assert hta.get_status(ws) == hta.OK
    ref, ref_lse, absv = P.tree_rows(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, c.ks, c.vs)
    P.check_attention(out, lse, ref, ref_lse, absv)
    out, lse = hta.prefix_attention_paged(q, c.kc, c.vc, c.table, c.prefix_len, workspace=ws, **c.paged())
    assert hta.get_status(ws) == hta.OK
    ref, ref_lse, absv = P.tree_rows(q, c.kc, c.vc, c.table, c.prefix_len, None, None, None, c.ks, c.vs)
    P.check_attention(out, lse, ref, ref_lse, absv)


def test_verify_q8_reports():
    for case, want in (("parent", hta.ERR_BAD_PARENT), ("len", hta.ERR_PREFIX_LEN_RANGE), ("block", hta.ERR_BAD_BLOCK)):
        c = Case([300, 40], [0, 0], 4, 2, 128, 16, True, seed=1)
        q, kt, vt = randn(2, 4, 7, 128, seed=1), randn(2, 2, 7, 128, seed=2), randn(2, 2, 7, 128, seed=3)
        parent = torch.tensor([[-1, 0, 1, 1, 0, 2, 5]] * 2, dtype=torch.int32).cuda()
        if case == "parent":
            parent[1, 3] = 3
        elif case == "len":
            c.prefix_len[1] = c.L_cap + 1
        else:
            c.table[1, 1] = -1
        ws = hta.new_q8_workspace(hta.Dims(2, 4, 2, 128, 7, c.L_cap, 0.0))
        out, lse = hta.verify_paged(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, workspace=ws, **c.paged())
        assert hta.get_status(ws) == want
        assert torch.isfinite(out[0].float()).all()
        if case != "block":
            assert torch.isnan(out[1].float()).all() and torch.isnan(lse[1]).all()


@pytest.mark.parametrize("bs", [16, 128])
def test_commit_q8(bs):
    Hkv, T, D = 3, 12, 128
    c = Case([0, 100, 31, 64], [5, 12, 4, 0], Hkv, Hkv, D, bs, True, seed=8)
    kt, vt = randn(4, Hkv, T, D, seed=1), randn(4, Hkv, T, D, seed=2)
    n = torch.tensor([5, 12, 13, 0], dtype=torch.int32).cuda()          # sequence 2: longer than the tree
    path = torch.stack([torch.randperm(T, generator=torch.Generator().manual_seed(b)).int() for b in range(4)]).cuda()
    ks, kc, vs, vc = c.ks.clone(), c.kc.clone(), c.vs.clone(), c.vc.clone()
    ws = status()
    hta.commit_paged(c.kc, c.vc, c.table, c.prefix_len, kt, vt, n, path, workspace=ws, **c.paged())
    assert hta.get_status(ws) == hta.ERR_BAD_PATH
    assert c.prefix_len.tolist() == [5, 112, 31, 64]
    for b in (0, 1):
        for d in range(int(n[b])):
            pos = c.pre[b] + d
            blk, at = int(c.table[b, pos // bs]), pos % bs
            for h in range(Hkv):
                for src, code, sc in ((kt, kc, ks), (vt, vc, vs)):
                    val, e = P.quantise_row(src[b, h, int(path[b, d])])
                    code[blk, h, at] = val.float().to(P.F8).cuda()
                    sc[blk, h, at] = e
    assert torch.equal(c.ks, ks) and torch.equal(c.vs, vs)
    assert torch.equal(c.kc.view(torch.uint8), kc.view(torch.uint8))
    assert torch.equal(c.vc.view(torch.uint8), vc.view(torch.uint8))


# ---------------------------------------------------------- a run of them all
@pytest.mark.parametrize("q8", [False, True])
def test_prompt_decode_verify_commit_run(q8):
    """A prompt rotated and written in two chunks, a decode step, then a tree
    verified, committed and read again, against one 64-bit attention over
    every key as it stands in the cache; the steps are captured in a graph
    and replayed."""
    Hq, Hkv, D, bs, T = 8, 2, 128, 16, 6
    total = 90
    c = Case([0], [total + T + 1], Hq, Hkv, D, bs, q8, seed=6)
    inv = freqs(D)
    q, k, v = randn(total, Hq, D, seed=1), randn(total, Hkv, D, seed=2), randn(total, Hkv, D, seed=3)
    pos = torch.arange(total, dtype=torch.int32, device="cuda")
    outs = torch.zeros_like(q)

    def prompt():
        for a, b in ((0, 50), (50, total - 1), (total - 1, total)):
            pre = torch.full((1,), a, dtype=torch.int32, device="cuda")
            start = torch.arange(0, 2 * (b - a), b - a, dtype=torch.int32, device="cuda")
            qr = hta.rope_append_paged(q[a:b], k[a:b], v[a:b], inv, c.kc, c.vc, c.table, pre, start, **c.paged())
            hta.chunk_attention_paged(qr, c.kc, c.vc, c.table, pre, start, out=outs[a:b], **c.paged())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        prompt()
    torch.cuda.current_stream().wait_stream(side)
    eager, kc0 = outs.clone(), c.kc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prompt()
    outs.zero_()
    c.kc.view(torch.uint8).fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs, eager)
    held = keys = P.keys_of(c.kc, c.ks, c.table, 0, 0, total, 0, bs)
    qr, _ = hta.qk_norm_rope(q, k, pos, inv)
    z, whole = torch.zeros(1, dtype=torch.int32).cuda(), torch.tensor([0, total], dtype=torch.int32).cuda()
    ref = P.chunk_rows(qr, c.kc, c.vc, c.table, z, whole, 0, c.ks, c.vs)
    for (t, h), (o, _, absv) in ref.items():
        bound = P.BF16 * o.abs() + (2 * P.BF16 + 3e-3) * absv
        assert ((P.cpu(outs[t, h]).double() - o).abs() <= bound).all()
    # the tree over the prompt, its accepted path committed and read by the next token
    qt, kt, vt = randn(1, Hq, T, D, seed=4), randn(1, Hkv, T, D, seed=5), randn(1, Hkv, T, D, seed=6)
    parent = torch.tensor([[-1, 0, 0, 1, 3, 2]], dtype=torch.int32).cuda()
    node = torch.tensor([[total, total + 1, total + 1, total + 2, total + 3, total + 2]], dtype=torch.int32).cuda()
    qt, kt = hta.qk_norm_rope(qt, kt, node, inv)
    L = torch.tensor([total], dtype=torch.int32).cuda()
    out, lse = hta.verify_paged(qt, c.kc, c.vc, c.table, L, kt, vt, parent, **c.paged())
    hta.commit_paged(c.kc, c.vc, c.table, L, kt, vt, torch.tensor([3], dtype=torch.int32).cuda(),
                     torch.tensor([[0, 1, 3, -1, -1, -1]], dtype=torch.int32).cuda(), **c.paged())
    assert L.tolist() == [total + 3]
    # node 3's row again, as a decode step over the committed path (its own key at position total + 2)
    one = torch.tensor([0, 1], dtype=torch.int32).cuda()
    again, _ = hta.chunk_attention_paged(qt[:, :, 3].contiguous(), c.kc, c.vc, c.table, L - 1, one, **c.paged())
    held = P.keys_of(c.vc, c.vs, c.table, 0, 0, total + 3, 0, bs)
    # the same row but for the tree keys' own rounding to the cache: bf16 none,
    # e4m3 moves three of 93 keys' scores and values by 2^-4 relative at most
    spread = float(held.abs().max())
    tol = (4 * P.BF16 + 6e-3 if not q8 else 0.1) * spread
    assert (again[0].float() - out[0, :, 3].float()).abs().max() <= tol


# ------------------------------------------------- what only bad values reach
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("Hq,new", [(8, 200), (4, 40), (2, 3)])
def test_masked_rows_may_hold_anything(q8, Hq, new):
    """An infinity or a NaN in the K or V of a token reaches the rows that see
    it (as NaN) and no other: not the earlier tokens of its chunk, not those
    whose window has passed it."""
    D, bs, pre, window = 128, 16, 150, 64
    c = Case([pre], [new], Hq, 2, D, bs, q8, seed=12)
    good = {w: c.attend(w)[0] for w in (0, window)}
    bad_at = pre + new // 2
    blk, at = int(c.table[0, bad_at // bs]), bad_at % bs
    for cache, scale, value in ((c.kc, c.ks, math.nan), (c.vc, c.vs, math.inf)):
        keep = (cache.clone(), None if scale is None else scale.clone())
        if q8:
            cache.view(torch.uint8)[blk, :, at] = 0x7f
            scale[blk, :, at] = 255
        else:
            cache[blk, :, at, 5] = value
        for w in (0, window):
            out, lse, code = c.attend(w)
            assert code == hta.OK
            sees = [pre + t >= bad_at and (w == 0 or pre + t - w < bad_at) for t in range(new)]
            for t in range(new):
                if sees[t]:
                    assert not torch.isfinite(out[t].float()).all(-1).any(), (t, w)
                else:
                    assert torch.equal(out[t], good[w][t]), (t, w)
        cache.copy_(keep[0])
        if q8:
            scale.copy_(keep[1])


@pytest.mark.parametrize("q8", [False, True])
def test_blocks_before_the_window_need_no_entry(q8):
    c = Case([500, 3], [20, 20], 8, 2, 128, 16, q8, seed=5)
    good, _, _ = c.attend(100)
    c.table[0, :(500 - 99) // 16] = -1                # wholly before every token's window
    out, _, code = c.attend(100)
    assert code == hta.OK and torch.equal(out, good)


def test_verify_q8_bad_tree_rows_reach_their_descendants_only():
    c = Case([200], [0], 4, 2, 128, 16, True, seed=1)
    T = 130
    q, kt, vt = randn(1, 4, T, 128, seed=1), randn(1, 2, T, 128, seed=2), randn(1, 2, T, 128, seed=3)
    parent = torch.tensor([[-1 if i < 4 else i - 4 for i in range(T)]], dtype=torch.int32).cuda()
    good, _ = hta.verify_paged(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, **c.paged())
    for t, value in ((kt, math.nan), (vt, math.inf), (vt, math.nan)):
        keep = t.clone()
        t[0, :, 9, 3] = value
        out, _ = hta.verify_paged(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, **c.paged())
        t.copy_(keep)
        for i in range(T):
            if i >= 9 and i % 4 == 1:
                assert not torch.isfinite(out[0, :, i].float()).all(-1).any(), i
            else:
                assert torch.equal(out[0, :, i], good[0, :, i]), i


# --------------------------------------------------------- sizes and schedules
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("pre,new,Hq,Hkv,D,bs", [
    ([700, 3, 40], [1, 1, 1], 16, 1, 128, 16), ([700, 3, 40], [1, 1, 1], 16, 1, 64, 32),
    ([100, 5, 1], [3, 1, 0], 8, 2, 64, 16), ([2000, 9], [1, 1], 3, 1, 128, 128), ([5] * 70, [1] * 70, 6, 2, 64, 16)])
def test_chunk_attention_few_rows(pre, new, Hq, Hkv, D, bs, q8):
    Case(pre, new, Hq, Hkv, D, bs, q8, seed=len(pre)).check()
    Case(pre, new, Hq, Hkv, D, bs, q8, seed=len(pre)).check(window=33)


@pytest.mark.parametrize("q8", [False, True])
def test_thousands_of_sequences(q8):
    """More sequences than the schedule keeps one by one."""
    g = torch.Generator().manual_seed(1)
    pre = torch.randint(0, 20, (2300,), generator=g).tolist()
    new = torch.randint(0, 3, (2300,), generator=g).tolist()
    c = Case(pre, new, 2, 1, 64, 16, q8, seed=3)
    rows = {(t, h) for t in range(0, c.N, 97) for h in (0, 1)}
    c.check(rows=rows)
    out, _, _ = c.attend()
    assert torch.isfinite(out.float()).all()


def test_no_tokens_at_all():
    c = Case([7, 3], [0, 0], 4, 2, 64, 16, seed=1)
    out, lse, code = c.attend()
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4) and code == hta.OK
    before = c.kc.clone()
    hta.append_paged(randn(0, 2, 64), randn(0, 2, 64), c.kc, c.vc, c.table, c.prefix_len, c.q_start, **c.paged())
    assert torch.equal(before.view(torch.uint8), c.kc.view(torch.uint8))


@pytest.mark.parametrize("q8", [False, True])
def test_a_captured_call_follows_the_lengths(q8):
    """Two graphs over one workspace, replayed after the lengths and the chunks
    on the device have changed, on another stream than the capture's."""
    c = Case([300, 40, 0], [30, 1, 70], 8, 2, 128, 32, q8, seed=8)
    ws = hta.new_chunk_workspace(c.q, c.kc, 3, L_cap=c.L_cap)
    out, lse = torch.zeros_like(c.q), torch.zeros(c.q.shape[:2], device="cuda")

    def call(window):
        hta.chunk_attention_paged(c.q, c.kc, c.vc, c.table, c.prefix_len, c.q_start, window=window, workspace=ws,
                                  out=out, lse=lse, **c.paged())
    call(0)
    torch.cuda.synchronize()
    graphs = []
    for window in (0, 50):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(window)
        graphs.append((g, window))
    side = torch.cuda.Stream()
    for pre, start in (([300, 40, 0], [0, 30, 31, 101]), ([290, 0, 7], [0, 2, 2, 40]), ([0, 40, 69], [0, 100, 100, 101])):
        c.prefix_len.copy_(torch.tensor(pre, dtype=torch.int32))
        c.q_start.copy_(torch.tensor(start, dtype=torch.int32))
        for g, window in graphs:
            want, want_lse, code = c.attend(window)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                g.replay()
            torch.cuda.current_stream().wait_stream(side)
            n = start[-1]
            assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_lse[:n])


def test_equal_calls_give_equal_bits():
    """Nothing depends on the order in which CTAs finish."""
    for q8 in (False, True):
        c = Case([4000, 100, 9], [5, 300, 1], 8, 2, 128, 64, q8, seed=2)
        first = c.attend()[:2]
        for _ in range(5):
            again = c.attend()[:2]
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


def test_wide_range_of_scales():
    """Rows of 1e-6 and of 1e3 in one e4m3 cache, K and V: each row's weight is
    right, whatever the others' scales."""
    for new, Hq in (([40], 4), ([1], 4), ([300], 2)):
        c = Case([260], new, Hq, 2, 128, 16, True, seed=3)
        for cache, scale in ((c.kc, c.ks), (c.vc, c.vs)):
            e = scale.int()
            live = e != 255
            g = torch.Generator(device="cuda").manual_seed(1)
            step = torch.randint(-20, 11 if scale is c.vs else 1, e.shape, generator=g, device="cuda")
            scale.copy_(torch.where(live, (e + step).clamp(16, 134), e).to(torch.uint8))
        c.check()


def test_workspaces_and_devices_are_checked():
    c = Case([40, 20], [4, 3], 4, 2, 64, 16, seed=3)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(hta.HtaError) as e:
        hta.chunk_attention_paged(c.q, c.kc, c.vc, c.table, c.prefix_len, c.q_start, workspace=small, **c.paged())
    assert e.value.code == hta.ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(hta.HtaError) as e:
        hta.append_paged(randn(7, 2, 64), randn(7, 2, 64), c.kc, c.vc, c.table, c.prefix_len, c.q_start,
                         workspace=small[:128], **c.paged())
    assert e.value.code == hta.ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(ValueError):
        hta.append_paged(randn(7, 2, 64).cpu(), randn(7, 2, 64), c.kc, c.vc, c.table, c.prefix_len, c.q_start, **c.paged())
    with pytest.raises(ValueError):
        hta.chunk_attention_paged(c.q, c.kc, c.vc, c.table, c.prefix_len.cpu(), c.q_start, **c.paged())
    with pytest.raises(hta.HtaError) as e:
        hta.chunk_attention_paged(c.q, c.kc, c.vc, c.table, c.prefix_len, c.q_start, window=-1, **c.paged())
    assert e.value.code == hta.ERR_INVALID_OPTION


def test_one_head_at_any_stride():
    """A single query head of wider rows; a single token of wider rows."""
    c = Case([50, 9], [7, 1], 1, 1, 128, 16, seed=4)
    want, want_lse, _ = c.attend()
    wide = torch.zeros((c.N, 4, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:3] = c.q
    c.q = wide[:, 2:3]
    out, lse, code = c.attend()
    assert code == hta.OK and torch.equal(out, want) and torch.equal(lse, want_lse)
    c.q = wide[:, 2].unsqueeze(1).transpose(0, 1).transpose(0, 1)
    assert torch.equal(c.attend()[0], want)
