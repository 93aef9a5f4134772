"""Padding tokens of an append through the C ABI: only the rows in front of
q_start[B] belong to the call (needs a B200)."""
import pytest
import torch

from tests.test_gpu_cache_ops import Case, freqs, randn, status
from tree_masked_verification_b200 import hta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("real", [[0, 0], [1, 0], [3, 40]])
def test_a_call_captured_for_more_tokens_than_there_are(real, rope, q8):
    """The token count of a launch is its largest; q_start says how many rows
    there are.  Same bytes as the call of that many tokens, nothing else
    written: the rows behind (here another tensor's) keep their NaN."""
    Hq, Hkv, D, n, most = 4, 2, 128, sum(real), 500
    a = Case([5, 60], real, Hq, Hkv, D, 16, q8, seed=3, pad=most - n)
    b = Case([5, 60], real, Hq, Hkv, D, 16, q8, seed=3, pad=most - n)
    qkv = randn(most, (Hq + 2 * Hkv) * D, seed=1)
    qkv[n:] = float("nan")
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    k, v = (qkv[:, i * D:(i + Hkv) * D].unflatten(1, (Hkv, D)) for i in (Hq, Hq + Hkv))
    out = torch.full((most, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    for c, rows in ((a, most), (b, n)):
        ws = status()
        args = (c.kc, c.vc, c.table, c.prefix_len, c.q_start)
        if rope:
            got = hta.rope_append_paged(q[:rows], k[:rows], v[:rows], freqs(D), *args, workspace=ws,
                                        q_out=out if rows == most else None, **c.paged())
        else:
            hta.append_paged(k[:rows], v[:rows], *args, workspace=ws, **c.paged())
        assert hta.get_status(ws) == hta.OK
    assert torch.equal(a.kc.view(torch.uint8), b.kc.view(torch.uint8))
    assert torch.equal(a.vc.view(torch.uint8), b.vc.view(torch.uint8))
    if q8:
        assert torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)
    if rope:
        assert torch.equal(out[:n], got) and (out[n:] == 9.0).all()
