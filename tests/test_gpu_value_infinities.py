"""Infinities and NaN in single values of V: the formula's result, column by
column, whether the key's tile is seen whole or in part (needs a B200)."""
import math

import pytest
import torch

from tests import cache_plain as P
from tests.test_gpu_cache_ops import Case, randn
from tree_masked_verification_b200 import hta

pytestmark = pytest.mark.gpu

# (column, value) of the keys that get one
BAD = [(0, math.inf), (5, -math.inf), (5, math.inf), (17, math.nan), (63, -math.inf), (40, math.inf)]


def check(got, ref, absv):
    """Infinities and NaN where the formula has them, the bound of the other
    tests elsewhere (a NaN's sign is not compared)."""
    got, ref = P.cpu(got).double(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]) and not torch.isinf(got[~inf]).any()
    ok = torch.isfinite(ref)
    bound = P.BF16 * ref.abs() + (2 * P.BF16 + 2 * (1e-4 + 128 * P.F32 * 32)) * absv * (1 + P.BF16)
    assert ((got - ref).abs() <= bound)[ok].all()


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pre,new,Hq", [([200], [1], 4), ([150], [40], 4), ([130], [200], 8), ([700] * 40, [30] * 40, 8)])
def test_chunk_columns(pre, new, Hq, D, window):
    """Keys in the prefix's whole tiles, at the border and among the chunk's own."""
    c = Case(pre, new, Hq, 2, D, 16, seed=D + new[0])
    keys = [3, pre[0] - 1, pre[0] - 60, pre[0] + new[0] // 2, pre[0] + new[0] - 1, pre[0] - 30]
    for b in (0, len(pre) - 1):
        for key, (col, value) in zip(keys, BAD):
            c.vc[int(c.table[b, key // 16]), b % 2, key % 16, col] = value
    rows = {(b * new[0] + t, h) for b in (0, len(pre) - 1) for t in range(0, new[0], 1 + new[0] // 20) for h in range(Hq)}
    rows |= {(b * new[0] + new[0] - 1, h) for b in (0, len(pre) - 1) for h in range(Hq)}
    out, lse, code = c.attend(window)
    assert code == hta.OK and torch.isfinite(lse).all()
    ref = P.chunk_rows(c.q, c.kc, c.vc, c.table, c.prefix_len, c.q_start, window, rows=rows)
    at = list(ref)
    check(out[[x[0] for x in at], [x[1] for x in at]], torch.stack([ref[x][0] for x in at]),
          torch.stack([ref[x][2] for x in at]))


@pytest.mark.parametrize("T,Hq,L,D", [(7, 2, 0, 64), (68, 4, 300, 128), (200, 4, 40, 128)])
def test_tree_columns_over_an_e4m3_cache(T, Hq, L, D):
    c = Case([L], [0], Hq, 2, D, 16, True, seed=T)
    q, kt, vt = randn(1, Hq, T, D, seed=1), randn(1, 2, T, D, seed=2), randn(1, 2, T, D, seed=3)
    for node, (col, value) in zip((0, 1, 4, 5, T // 2, T - 1), BAD):
        vt[0, node % 2, node, col] = value
    parent = torch.tensor([[-1 if i < 4 else i - 4 for i in range(T)]], dtype=torch.int32).cuda()
    ws = hta.new_q8_workspace(hta.Dims(1, Hq, 2, D, T, c.L_cap, 0.0))
    out, lse = hta.verify_paged(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, workspace=ws, **c.paged())
    assert hta.get_status(ws) == hta.OK and torch.isfinite(lse).all()
    ref, _, absv = P.tree_rows(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, c.ks, c.vs)
    check(out, ref, absv)


def same_or_nan(got, got_lse, ref, ref_lse, absv):
    """Rows of a finite lse within the bound, the others NaN."""
    ok = torch.isfinite(ref_lse)
    assert ok.any() and not ok.all()
    P.check_attention(got[ok], got_lse[ok], ref[ok], ref_lse[ok], absv[ok])
    assert torch.isnan(P.cpu(got)[~ok].float()).all() and torch.isnan(P.cpu(got_lse)[~ok]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pre,new,Hq", [([200], [1], 16), ([150], [40], 4), ([130], [200], 8)])
def test_infinite_keys(pre, new, Hq, D):
    """A key with an infinity: weight 0 for queries whose score it makes -inf,
    NaN for those whose score it makes +inf."""
    c = Case(pre, new, Hq, 2, D, 16, seed=D + new[0])
    for key in (3, pre[0] + new[0] // 2):
        c.kc[int(c.table[0, key // 16]), :, key % 16, 7] = math.inf
    c.q[:, ::2, 7] = -c.q[:, ::2, 7].abs() - 0.01
    c.q[:, 1::2, 7] = c.q[:, 1::2, 7].abs() + 0.01
    out, lse, code = c.attend()
    assert code == hta.OK
    ref = P.chunk_rows(c.q, c.kc, c.vc, c.table, c.prefix_len, c.q_start)
    at = list(ref)
    i, h = [x[0] for x in at], [x[1] for x in at]
    same_or_nan(out[i, h], lse[i, h], torch.stack([ref[x][0] for x in at]),
                torch.tensor([ref[x][1] for x in at], dtype=torch.float64), torch.stack([ref[x][2] for x in at]))


@pytest.mark.parametrize("T,Hq,L,D", [(68, 4, 300, 128), (200, 4, 40, 64)])
def test_infinite_tree_keys_over_an_e4m3_cache(T, Hq, L, D):
    c = Case([L], [0], Hq, 2, D, 16, True, seed=T)
    q, kt, vt = randn(1, Hq, T, D, seed=1), randn(1, 2, T, D, seed=2), randn(1, 2, T, D, seed=3)
    q[:, :, ::2, 7] = -q[:, :, ::2, 7].abs() - 0.01
    q[:, :, 1::2, 7] = q[:, :, 1::2, 7].abs() + 0.01
    kt[0, :, 1, 7] = math.inf
    kt[0, :, 8, 7] = math.inf
    parent = torch.tensor([[-1 if i < 4 else i - 3 for i in range(T)]], dtype=torch.int32).cuda()
    out, lse = hta.verify_paged(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, **c.paged())
    ref, ref_lse, absv = P.tree_rows(q, c.kc, c.vc, c.table, c.prefix_len, kt, vt, parent, c.ks, c.vs)
    same_or_nan(out, lse, ref, ref_lse, absv)
