"""Chunk attention over bf16 caches where few keys take most of a row's weight:
the rounding of the weights for the tensor cores must not reach the result of
a row that one key dominates (needs a B200)."""
import math

import pytest
import torch

from tests import cache_plain as P
from tests.test_gpu_cache_ops import Case, randn

pytestmark = pytest.mark.gpu


def check_rows(c, window, rows):
    """The weights w_j are rounded to bf16, w_j (1 + d_j) with |d_j| <= u = 2^-8, and
    divided by their own sum:
      out - ref = sum p_j d_j (v_j - ref) / (1 + sum p_j d_j),
    which is at most u (1 + 2u) sum p_j |v_j - ref|.  The output's rounding is half a
    step of bf16 at the result, 2^(e - 9) for 2^(e - 1) <= |result| < 2^e.  Scores are
    fp32 sums of D products, D 2^-24 of the sum of their sizes at most, and exponentials
    good to 1e-4: twice that, for a weight and for the sum it is divided by."""
    out, lse, code = c.attend(window)
    assert code == 0
    u, G, D = P.BF16, c.Hq // c.Hkv, c.D
    start = c.q_start.tolist()
    q, out, lse = P.cpu(c.q).double(), P.cpu(out).double(), P.cpu(lse).double()
    worst = -math.inf
    for b in range(len(c.pre)):
        n = c.pre[b] + c.new[b]
        for h in range(c.Hkv):
            blocks = c.table[b, :-(-n // c.bs)].long()
            k, v = (P.cpu(x[blocks, h].reshape(-1, D)[:n]).double() for x in (c.kc, c.vc))
            for t in range(start[b], start[b + 1]):
                if t not in rows:
                    continue
                pos = c.pre[b] + t - start[b]
                lo = max(0, pos - window + 1) if window else 0
                kk, vv = k[lo:pos + 1], v[lo:pos + 1]
                for i in range(h * G, h * G + G):
                    s = kk @ q[t, i] / math.sqrt(D)
                    soft = 1e-4 + D * P.F32 * float((kk.abs() @ q[t, i].abs()).max()) / math.sqrt(D)
                    m = torch.logsumexp(s, 0)
                    p = torch.exp(s - m)
                    ref = p @ vv
                    before = u * (1 + 2 * u) * (p @ (vv - ref).abs()) + 2 * soft * (p @ vv.abs())
                    half = torch.pow(2.0, torch.frexp(ref.abs() + before).exponent.double() - 9)
                    worst = max(worst, float(((out[t, i] - ref).abs() - before - half).max()))
                    assert abs(float(lse[t, i] - m)) <= soft + 1e-5
    assert worst <= 0, worst


# Many sequences, so that a CTA takes more than a tile or two of an item: the
# running maximum of several tiles is what makes weights above one.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,Hq", [(1, 32), (30, 16), (40, 32)])
@pytest.mark.parametrize("sharp,window", [(3.0, 0), (8.0, 0), (8.0, 700)])
def test_peaked_rows(new, Hq, D, sharp, window):
    c = Case([900] * 16, [new] * 16, Hq, 8, D, 32, seed=new + D)
    c.q *= sharp
    check_rows(c, window, set(range(0, c.N, 1 + c.N // 24)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,Hq", [(1, 8), (16, 8), (40, 16)])
def test_the_later_of_two_keys(new, Hq, D):
    """A key of the first tile, then one of the third with up to 2^8 times its
    weight (within the running maximum's slack), and V of the first 0."""
    B = 40
    c = Case([700] * B, [new] * B, Hq, 4, D, 16, seed=D + new)
    u = randn(D, seed=2).float()
    u = (u / u.norm() * math.sqrt(D)).to(torch.bfloat16)
    c.kc.copy_(torch.where(torch.isnan(c.kc), c.kc, -u * 4))             # all others: far below
    first, second = c.table[:, 0].long(), c.table[:, 270 // 16].long()
    c.vc[first, :, 5] = 0
    c.kc[first, :, 5] = 0
    c.kc[second, :, 270 % 16] = u
    steps = torch.linspace(1.0, 5.4, c.N * Hq).view(c.N, Hq, 1).cuda()
    c.q = (u.float() * steps / math.sqrt(D)).to(torch.bfloat16)
    check_rows(c, 0, set(range(0, c.N, 1 + c.N // 60)))
