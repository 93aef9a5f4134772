"""e4m3 caches whose rows' scales lie far apart, over the whole range of the
scale byte, against the plain 64-bit forms (needs a B200).  A row's result may
depend on the rows it sees alone, and on those by their weights."""
import pytest
import torch

from tests import cache_plain as P
from tests.test_gpu_cache_ops import Case, randn
from tree_masked_verification_b200 import hta

pytestmark = pytest.mark.gpu

# (tokens, Hq): few rows, one row tile an item, two row tiles (2 KV heads)
ROWS = [(3, 4), (20, 8), (150, 8)]


def at_keys(c, b, keys):
    """(block, place) of the keys of sequence b."""
    blk = c.table[b, torch.tensor(keys).cuda() // c.bs].long()
    return blk, torch.tensor(keys).cuda() % c.bs


def own_values(c, b, t, h):
    """V of token t (its own key), head h, as the cache holds it."""
    blk, at = at_keys(c, b, [c.pre[b] + t])
    return c.vc[blk[0], h, at[0]].double() * 2.0 ** (int(c.vs[blk[0], h, at[0]]) - 127)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,Hq", ROWS)
def test_a_window_of_one_returns_the_own_row(new, Hq, D):
    """Softmax over one key: the result is its V row, to the bit (four
    significant bits fit bf16), whatever scales stand beside it."""
    c = Case([37], [new], Hq, 2, D, 16, True, seed=D + new)
    live = c.vs != 255
    g = torch.Generator(device="cuda").manual_seed(7)
    for s in (c.ks, c.vs):
        e = torch.randint(16 if s is c.vs else 90, 135 if s is c.vs else 121, s.shape, generator=g, device="cuda")
        s.copy_(torch.where(live, e, s.int()).to(torch.uint8))
    out, lse, code = c.attend(1)
    assert code == hta.OK
    for t in range(new):
        for h in range(Hq):
            assert torch.equal(out[t, h].double(), own_values(c, 0, t, h // (Hq // 2))), (t, h)


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("least", [16, 60, 102])
@pytest.mark.parametrize("new,Hq", ROWS)
def test_scales_over_the_whole_range(new, Hq, least, window):
    """Every V row a scale of its own; the first token of a prompt sees itself
    alone, the others keys of any scale, none of them the tile's largest for sure."""
    for pre in (0, 300):
        c = Case([pre], [new], Hq, 2, 128, 16, True, seed=least)
        g = torch.Generator(device="cuda").manual_seed(least)
        e = torch.randint(least, 135, c.vs.shape, generator=g, device="cuda")
        c.vs.copy_(torch.where(c.vs != 255, e, c.vs.int()).to(torch.uint8))
        c.check(window)


@pytest.mark.parametrize("k", [5, 14, 20, 26, 60])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,Hq", ROWS)
def test_large_values_of_hardly_any_weight(new, Hq, D, k):
    """V rows 2^k above all others among the first keys: hidden by a window, or
    seen with scores far below the others'.  What is left is the others' average."""
    pre = 700
    c = Case([pre], [new], Hq, 2, D, 32, True, seed=k + new)
    c.vs.copy_(torch.where(c.vs != 255, 72, c.vs.int()).to(torch.uint8))
    blk, at = at_keys(c, 0, list(range(3, 9)))
    c.vs[blk, :, at] = 72 + k
    c.check(window=500)
    u = randn(D, seed=1).float()
    c.q = (c.q.float() * 0.5 + u).to(torch.bfloat16)
    codes, e = Case.quantise((-u * 24).to(torch.bfloat16)[None])       # scores of about -24 sqrt(D)
    c.kc[blk, :, at], c.ks[blk, :, at] = codes[0], e[0]
    c.check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,Hq", ROWS)
def test_a_zero_value_that_takes_most_of_the_weight(new, Hq, D):
    """Keys that take most of the weight and hold V rows of zeros (the least scale)."""
    c = Case([400], [new], Hq, 2, D, 64, True, seed=new)
    u = randn(D, seed=1).float()
    c.q = (c.q.float() * 0.5 + u).to(torch.bfloat16)
    blk, at = at_keys(c, 0, [0, 1, 200])
    codes, e = Case.quantise((u * 0.5).to(torch.bfloat16)[None])
    c.kc[blk, :, at], c.ks[blk, :, at] = codes[0], e[0]
    c.vc.view(torch.uint8)[blk, :, at] = 0
    c.vs[blk, :, at] = 16
    c.check()


@pytest.mark.parametrize("new,Hq", ROWS)
def test_keys_of_scales_far_apart(new, Hq):
    """K rows so small that they need queries of a hundred thousand beside rows
    of the largest scale, which a window hides or whose scores are far below."""
    c = Case([300], [new], Hq, 2, 128, 16, True, seed=new)
    u = randn(128, seed=1).float()
    c.q = ((c.q.float() + u) * 2.0 ** 17).to(torch.bfloat16)
    c.ks.copy_(torch.where(c.ks != 255, (c.ks.int() - 17).clamp(min=16), c.ks.int()).to(torch.uint8))
    blk, at = at_keys(c, 0, [1, 290])
    codes, _ = Case.quantise((-u).to(torch.bfloat16)[None])
    c.kc[blk, :, at], c.ks[blk, :, at] = codes[0], 134
    for window in (0, 5):
        ref = P.chunk_rows(c.q, c.kc, c.vc, c.table, c.prefix_len, c.q_start, window, c.ks, c.vs)
        out, lse, code = c.attend(window)
        assert code == hta.OK
        i = list(ref)
        t, h = [x[0] for x in i], [x[1] for x in i]
        P.check_attention(out[t, h], lse[t, h], torch.stack([ref[x][0] for x in i]),
                          torch.tensor([ref[x][1] for x in i], dtype=torch.float64), torch.stack([ref[x][2] for x in i]),
                          scores=64.0)


@pytest.mark.parametrize("T,Hq,L", [(5, 2, 0), (68, 2, 0), (68, 8, 300), (130, 2, 300), (200, 4, 40)])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_rows_of_scales_far_apart(T, Hq, L, D):
    """Tree rows of sizes from 1e-12 to 1e6: a node's result comes from its
    own path and the prefix, whatever the other branches hold."""
    c = Case([L], [0], Hq, 2, D, 16, True, seed=T)
    g = torch.Generator().manual_seed(T)
    q, kt, vt = randn(1, Hq, T, D, seed=1), randn(1, 2, T, D, seed=2), randn(1, 2, T, D, seed=3)
    size = torch.pow(10.0, torch.randint(-12, 7, (1, 2, T, 1), generator=g).float()).cuda()
    vt = (vt.float() * size).to(torch.bfloat16)
    kt = (kt.float() * torch.pow(2.0, -torch.randint(0, 40, (1, 2, T, 1), generator=g).float()).cuda()).to(torch.bfloat16)
    vt[:, :, 2] = 0
    kt[:, :, 3] = 0
    parent = torch.tensor([[-1 if i < 4 or i % 11 == 0 else int(torch.randint(max(0, i - 9), i, (1,), generator=g))
                            for i in range(T)]], dtype=torch.int32).cuda()
    ws = hta.new_q8_workspace(hta.Dims(1, Hq, 2, D, T, c.L_cap, 0.0))
    out, lse = hta.verify_paged(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, workspace=ws, **c.paged())
    assert hta.get_status(ws) == hta.OK
    ref, ref_lse, absv = P.tree_rows(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, c.ks, c.vs)
    P.check_attention(out, lse, ref, ref_lse, absv)


def test_one_cache_gives_one_answer_whatever_the_row_count():
    """The last token of a chunk, alone and at the end of its chunk."""
    c = Case([290], [60], 4, 2, 128, 16, True, seed=3)
    g = torch.Generator(device="cuda").manual_seed(3)
    e = torch.randint(70, 135, c.vs.shape, generator=g, device="cuda")
    c.vs.copy_(torch.where(c.vs != 255, e, c.vs.int()).to(torch.uint8))
    out, lse, _ = c.attend()
    ref = P.chunk_rows(c.q, c.kc, c.vc, c.table, c.prefix_len, c.q_start, 0, c.ks, c.vs,
                       rows={(59, h) for h in range(4)})
    one = torch.tensor([0, 1], dtype=torch.int32).cuda()
    alone, alone_lse = hta.chunk_attention_paged(c.q[59:].contiguous(), c.kc, c.vc, c.table, c.prefix_len + 59, one,
                                                 **c.paged())
    for got, got_lse in ((out[59], lse[59]), (alone[0], alone_lse[0])):
        P.check_attention(got, got_lse, torch.stack([ref[(59, h)][0] for h in range(4)]),
                          torch.tensor([ref[(59, h)][1] for h in range(4)], dtype=torch.float64),
                          torch.stack([ref[(59, h)][2] for h in range(4)]))


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("new,Hq", ROWS)
def test_a_nan_row_beside_scales_far_apart(new, Hq, window):
    """A row held as NaN reaches the rows that see it and no other, in tiles
    whose rows keep their own scales too; so do bytes behind the last key."""
    pre = 150
    c = Case([pre], [new], Hq, 2, 128, 16, True, seed=12)
    g = torch.Generator(device="cuda").manual_seed(2)
    for s, lo, hi in ((c.ks, 90, 120), (c.vs, 40, 135)):
        e = torch.randint(lo, hi, s.shape, generator=g, device="cuda")
        s.copy_(torch.where(s != 255, e, torch.randint(0, 256, s.shape, generator=g, device="cuda")).to(torch.uint8))
    c.check(window)
    good, _, _ = c.attend(window)
    bad_at = pre + new // 2
    blk, at = at_keys(c, 0, [bad_at])
    for cache, scale in ((c.kc, c.ks), (c.vc, c.vs)):
        keep = cache.clone(), scale.clone()
        cache.view(torch.uint8)[blk, :, at] = 0x7f
        scale[blk, :, at] = 255
        out, lse, code = c.attend(window)
        assert code == hta.OK
        for t in range(new):
            if pre + t >= bad_at and (window == 0 or pre + t - window < bad_at):
                assert torch.isnan(out[t].float()).all() and torch.isnan(lse[t]).all(), t
            else:
                assert torch.equal(out[t], good[t]), t
        cache.copy_(keep[0])
        scale.copy_(keep[1])


# -------------------------------------------- several tiles of an item in one CTA
MANY = [(2, 16), (30, 16), (40, 16)]            # few rows; one row tile; two (4 KV heads)


def many(new, Hq, D, seed):
    """Enough sequences that a CTA takes whole items: references carried from
    tile to tile, not joined from partials.  And the rows to look at."""
    c = Case([700] * 60, [new] * 60, Hq, 4, D, 32, True, seed=seed)
    rows = {(b * new + t, h) for b in (0, 7, 30, 59) for t in {0, new // 2, new - 1} for h in (0, Hq // 2, Hq - 1)}
    return c, rows


@pytest.mark.parametrize("k", [6, 14, 20, 26, 60])
@pytest.mark.parametrize("new,Hq", MANY)
@pytest.mark.parametrize("D", [64, 128])
def test_large_values_of_hardly_any_weight_many(new, Hq, D, k):
    c, rows = many(new, Hq, D, k + new)
    c.vs.copy_(torch.where(c.vs != 255, 70, c.vs.int()).to(torch.uint8))
    first = c.table[:, 0].long()
    c.vs[first, :, 3:9] = 70 + k
    c.check(window=600, rows=rows)
    u = randn(D, seed=1).float()
    c.q = (c.q.float() * 0.5 + u).to(torch.bfloat16)
    codes, e = Case.quantise((-u * 24).to(torch.bfloat16)[None])
    for at in range(3, 9):
        c.kc[first, :, at], c.ks[first, :, at] = codes[0], e[0]
    c.check(rows=rows)
    third = c.table[:, 9].long()                        # the same, met last
    c.vs[first, :, 3:9] = 70
    c.vs[third, :, 5] = 70 + k
    c.kc[third, :, 5], c.ks[third, :, 5] = codes[0], e[0]
    c.check(rows=rows)


@pytest.mark.parametrize("new,Hq", MANY)
@pytest.mark.parametrize("D", [64, 128])
def test_tiles_of_falling_and_rising_scales(new, Hq, D):
    """Whole tiles of scales from the least to the largest, in both orders, rows
    within a tile alike or not; a first tile of zeros that takes most of the weight."""
    for mode in ("falls", "rises", "random", "zeros"):
        c, rows = many(new, Hq, D, len(mode))
        n = c.table.shape[1] - 1                         # blocks of 32 keys: four to a tile
        for j in range(n):
            blk = c.table[:, j].long()
            blk = blk[blk >= 0]
            tile = j // 4
            if mode == "zeros":
                if tile == 0:
                    c.vc.view(torch.uint8)[blk] = 0
                    c.vs[blk] = 16
                continue
            e = {"falls": 130 - 20 * tile, "rises": 20 + 18 * tile, "random": (37 * (tile + 1)) % 115 + 18}[mode]
            c.vs[blk] = torch.where(c.vs[blk] != 255, e, 255).to(torch.uint8)
        if mode == "zeros":
            u = randn(D, seed=1).float()
            c.q = (c.q.float() * 0.5 + u).to(torch.bfloat16)
            codes, e = Case.quantise((u * 0.4).to(torch.bfloat16)[None])
            blk = c.table[:, 0].long()
            c.kc[blk, :, 7], c.ks[blk, :, 7] = codes[0], e[0]
        c.check(rows=rows)
        c.check(window=300, rows=rows)


@pytest.mark.parametrize("new,Hq", MANY)
def test_scales_over_the_whole_range_many(new, Hq):
    for lk, lv in ((90, 18), (16, 110)):
        c, rows = many(new, Hq, 128, lk)
        g = torch.Generator(device="cuda").manual_seed(lk)
        for s, lo, hi in ((c.ks, lk, 121), (c.vs, lv, 135)):
            e = torch.randint(lo, hi, s.shape, generator=g, device="cuda")
            s.copy_(torch.where(s != 255, e, s.int()).to(torch.uint8))
        c.check(rows=rows)
        c.check(window=200, rows=rows)


@pytest.mark.parametrize("T,D", [(5, 128), (68, 64), (150, 128)])
def test_trees_over_many_sequences_of_scales_far_apart(T, D):
    """Trees over prefixes of several tiles: the prefix's scales and the tree's."""
    B, Hq, Hkv = 24, 8, 8
    c = Case([500] * B, [0] * B, Hq, Hkv, D, 32, True, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T)
    for s, lo, hi in ((c.ks, 100, 121), (c.vs, 40, 135)):
        e = torch.randint(lo, hi, s.shape, generator=g, device="cuda")
        s.copy_(torch.where(s != 255, e, s.int()).to(torch.uint8))
    h = torch.Generator().manual_seed(T)
    q, kt, vt = randn(B, Hq, T, D, seed=1), randn(B, Hkv, T, D, seed=2), randn(B, Hkv, T, D, seed=3)
    vt = (vt.float() * torch.pow(10.0, torch.randint(-9, 4, (B, Hkv, T, 1), generator=h).float()).cuda()).to(torch.bfloat16)
    parent = torch.tensor([[-1 if i < 4 else i - 1 - i % 4 for i in range(T)]] * B, dtype=torch.int32).cuda()
    ws = hta.new_q8_workspace(hta.Dims(B, Hq, Hkv, D, T, c.L_cap, 0.0))
    out, lse = hta.verify_paged(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, workspace=ws, **c.paged())
    assert hta.get_status(ws) == hta.OK
    for b in (0, 11, 23):
        i = slice(b, b + 1)
        ref, ref_lse, absv = P.tree_rows(q[i, :2], c.kc[:, :2], c.vc[:, :2], c.table[i], c.prefix_len[i], kt[i, :2],
                                         vt[i, :2], parent[i], c.ks[:, :2], c.vs[:, :2])
        P.check_attention(out[i, :2], lse[i, :2], ref, ref_lse, absv)
