"""Calls on a stream of the caller's that allocate their results and their
workspace themselves (needs a B200)."""
import pytest
import torch

from tests.test_gpu_cache_ops import Case, freqs, randn
from tree_masked_verification_b200 import hta

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, T, BS = 2, 8, 2, 128, 6, 16


def calls():
    """name -> (a call that takes stream=, what it wrote)"""
    parent = torch.tensor([[-1, 0, 0, 1, 1, 2]] * B, dtype=torch.int32).cuda()
    q, kt, vt = randn(B, HQ, T, D, seed=1), randn(B, HKV, T, D, seed=2), randn(B, HKV, T, D, seed=3)
    kp, vp = randn(B, HKV, 96, D, seed=4), randn(B, HKV, 96, D, seed=5)
    kr, vr = randn(B, HKV, 128, D, seed=4), randn(B, HKV, 128, D, seed=5)
    L = torch.tensor([90, 40], dtype=torch.int32).cuda()
    got = {
        "verify": lambda s: hta.verify(q, kp, vp, L, kt, vt, parent, stream=s),
        "prefix_attention": lambda s: hta.prefix_attention(q, kp, vp, L, stream=s),
        "window_verify": lambda s: hta.window_verify(q, kr, vr, L, kt, vt, parent, stream=s),
        "tree_mask": lambda s: (hta.tree_mask(parent, stream=s),),
        "tree_partial": lambda s: hta.tree_partial(q, kt, vt, parent, stream=s),
        "prefix_partial": lambda s: hta.prefix_partial(q, kp, vp, L, stream=s)[:2],
    }
    logits, draft = randn(B, T + 1, 50, seed=6), torch.zeros(B, T, dtype=torch.int32).cuda()
    got["accept_greedy"] = lambda s: hta.accept_greedy(logits, draft, parent, stream=s)
    n = torch.tensor([2, 1], dtype=torch.int32).cuda()
    path = torch.tensor([[0, 1, -1, -1, -1, -1], [0, -1, -1, -1, -1, -1]], dtype=torch.int32).cuda()

    def commit(s):
        k, v, pre = kp.clone(), vp.clone(), torch.tensor([50, 40], dtype=torch.int32).cuda()
        torch.cuda.synchronize()
        hta.commit(k, v, pre, kt, vt, n, path, stream=s)
        return k, v, pre
    got["commit"] = commit
    for q8 in (False, True):
        c = Case([60, 33], [9, 1], HQ, HKV, D, BS, q8, seed=7)
        k, v = randn(10, HKV, D, seed=8), randn(10, HKV, D, seed=9)
        args = (c.kc, c.vc, c.table, c.prefix_len)
        for x in args[:2] + (() if c.ks is None else (c.ks, c.vs)):     # (NaN in unused rows compares unequal)
            x.view(torch.uint8).copy_(torch.where(x.view(torch.uint8) == 255, 0, x.view(torch.uint8)))
        w = "-q8" if q8 else ""
        got.update({
            "verify_paged" + w: lambda s, c=c, a=args: hta.verify_paged(q, *a, kt, vt, parent, stream=s, **c.paged()),
            "prefix_attention_paged" + w: lambda s, c=c, a=args: hta.prefix_attention_paged(q, *a, stream=s, **c.paged()),
            "chunk_attention_paged" + w: lambda s, c=c, a=args: hta.chunk_attention_paged(c.q, *a, c.q_start, stream=s,
                                                                                         **c.paged()),
            "rope_append_paged" + w: lambda s, c=c, a=args: (hta.rope_append_paged(
                c.q, k, v, freqs_, *a, c.q_start, stream=s, **c.paged()), c.kc.view(torch.uint8)),
            "append_paged" + w: lambda s, c=c, a=args: (hta.append_paged(k, v, *a, c.q_start, stream=s, **c.paged()),
                                                        c.kc.view(torch.uint8))[1:],
            "commit_paged" + w: lambda s, c=c, a=args: (hta.commit_paged(
                *a, kt, vt, zero_, path, stream=s, **c.paged()), c.kc.view(torch.uint8))[1:],
        })
    freqs_, zero_ = freqs(D), torch.zeros(B, dtype=torch.int32).cuda()
    pos = torch.arange(10, dtype=torch.int32).cuda()
    q3, k3 = randn(10, HQ, D, seed=1), randn(10, HKV, D, seed=2)
    got["qk_norm_rope"] = lambda s: hta.qk_norm_rope(q3, k3, pos, freqs_, stream=s)
    return got


NAMES = ["verify", "prefix_attention", "window_verify", "tree_mask", "tree_partial", "prefix_partial", "accept_greedy",
         "commit", "qk_norm_rope"] + [n + w for w in ("", "-q8") for n in (
             "verify_paged", "prefix_attention_paged", "chunk_attention_paged", "rope_append_paged", "append_paged",
             "commit_paged")]


@pytest.fixture(scope="module")
def table():
    torch.cuda.synchronize()
    t = calls()
    assert sorted(t) == sorted(NAMES)
    torch.cuda.synchronize()
    return t


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_allocates_belongs_to_its_stream(name, as_handle, table, monkeypatch):
    """Every tensor that the binding makes on the way is made with the call's
    stream current, so that it is filled in that stream's order and freed to it."""
    side = torch.cuda.Stream()
    seen = []
    for make in ("empty", "empty_like", "zeros"):
        real = getattr(torch, make)

        def spy(*a, real=real, **kw):
            t = real(*a, **kw)
            if t.is_cuda:
                seen.append(torch.cuda.current_stream().cuda_stream)
            return t
        monkeypatch.setattr(hta.torch, make, spy)
    want = table[name](torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [w.clone() for w in want]
    torch.cuda.synchronize()
    seen.clear()
    got = table[name](side.cuda_stream if as_handle else side)
    assert all(s == side.cuda_stream for s in seen) and (seen or name.startswith("chunk")), (seen, side.cuda_stream)
    side.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_a_result_outlives_its_stream_s_next_calls(table):
    """A result dropped while the current stream still reads it is not handed
    to the side stream's next call."""
    side = torch.cuda.Stream()
    call = table["chunk_attention_paged"]
    out, lse = call(side)
    side.synchronize()
    want = out.clone()
    held = torch.empty_like(out)
    torch.cuda._sleep(200_000_000)                       # the current stream: a tenth of a second behind
    held.copy_(out)
    del out, lse
    for _ in range(4):
        other, _ = call(side)
        with torch.cuda.stream(side):
            other.fill_(7.0)
        del other
    torch.cuda.synchronize()
    assert torch.equal(held, want)
