"""Refusals of the calls on new tokens and e4m3 caches, all on the host, and
the plain forms the GPU tests compare with (no GPU needed)."""
import ctypes
import math

import pytest
import torch

from tests import cache_plain as P
from tree_masked_verification_b200 import build, hta

BF16 = torch.bfloat16
WS, WS_BYTES = 4096 * 90, 1 << 30


@pytest.fixture(scope="module")
def lib():
    build.build()
    return hta.load()


def heads(p=4096, b=0, t=1024, h=128):
    return hta._heads_struct(p, b, t, h)


def rope(**kw):
    d = dict(inv_freq=4096 * 7, rot_dim=128, interleaved=0, scale=1.0, q_weight=None, k_weight=None, eps=1e-6)
    d.update(kw)
    return hta.Rope(*d.values())


def cache(**kw):
    d = dict(k_cache=4096 * 30, v_cache=4096 * 31, block_table=4096 * 32, num_blocks=64, block_size=16, max_blocks=64,
             k_scale=None, v_scale=None)
    d.update(kw)
    return hta.Cache(*d.values())


def dims(**kw):
    d = dict(B=2, Hq=8, Hkv=2, D=128, T=10, L_cap=1024, scale=0.0)
    d.update(kw)
    return hta.Dims(*d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), hta.ERR_UNSUPPORTED_D), (dict(T=-1), hta.ERR_INVALID_DIMS), (dict(Hq=0), hta.ERR_INVALID_DIMS),
    (dict(B=1 << 16, T=1 << 16), hta.ERR_INVALID_DIMS), (dict(rope=rope(rot_dim=3)), hta.ERR_INVALID_OPTION),
    (dict(rope=rope(rot_dim=130)), hta.ERR_INVALID_OPTION), (dict(rope=rope(rot_dim=0)), hta.ERR_INVALID_OPTION),
    (dict(rope=rope(eps=-1.0)), hta.ERR_INVALID_OPTION), (dict(rope=rope(eps=math.nan)), hta.ERR_INVALID_OPTION),
    (dict(rope=rope(scale=-1.0)), hta.ERR_INVALID_OPTION), (dict(rope=rope(scale=math.inf)), hta.ERR_INVALID_OPTION),
    (dict(rope=rope(inv_freq=None)), hta.ERR_NULL_POINTER), (dict(rope=rope(inv_freq=4098)), hta.ERR_MISALIGNED),
    (dict(rope=rope(q_weight=4104)), hta.ERR_MISALIGNED), (dict(rope=None), hta.ERR_NULL_POINTER),
    (dict(q=None), hta.ERR_NULL_POINTER), (dict(q=heads(p=0)), hta.ERR_NULL_POINTER),
    (dict(k=heads(p=4104)), hta.ERR_MISALIGNED), (dict(k=heads(t=1028)), hta.ERR_MISALIGNED),
    (dict(qo=heads(h=4)), hta.ERR_MISALIGNED), (dict(pos=None), hta.ERR_NULL_POINTER),
    (dict(pos=4097), hta.ERR_MISALIGNED), (dict(T=0, q=None), hta.OK), (dict(B=0), hta.OK)])
def test_norm_rope_refusals(lib, kw, code):
    a = dict(B=1, T=4, Hq=8, Hkv=2, D=128, q=heads(), k=heads(4096 * 2), pos=4096 * 3, rope=rope(), qo=heads(4096 * 4),
             ko=heads(4096 * 5))
    a.update(kw)
    assert lib.longspec_hta_qk_norm_rope(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(d=dims(D=32)), hta.ERR_UNSUPPORTED_D), (dict(d=dims(Hq=7)), hta.ERR_INVALID_DIMS),
    (dict(d=dims(T=-1)), hta.ERR_INVALID_DIMS), (dict(d=dims(L_cap=1025)), hta.ERR_INVALID_DIMS),
    (dict(c=cache(block_size=24)), hta.ERR_INVALID_DIMS), (dict(c=cache(num_blocks=0)), hta.ERR_INVALID_DIMS),
    (dict(c=cache(num_blocks=1 << 27)), hta.ERR_INVALID_DIMS), (dict(c=None), hta.ERR_NULL_POINTER),
    (dict(c=cache(k_cache=None)), hta.ERR_NULL_POINTER), (dict(c=cache(block_table=None)), hta.ERR_NULL_POINTER),
    (dict(c=cache(v_cache=4096 + 8)), hta.ERR_MISALIGNED), (dict(c=cache(k_scale=4096)), hta.ERR_INVALID_OPTION),
    (dict(c=cache(k_scale=4096, v_scale=4104)), hta.ERR_MISALIGNED), (dict(pre=None), hta.ERR_NULL_POINTER),
    (dict(start=4098), hta.ERR_MISALIGNED), (dict(k=heads(p=0)), hta.ERR_NULL_POINTER),
    (dict(v=heads(t=1030)), hta.ERR_MISALIGNED), (dict(ws=None), hta.ERR_NULL_POINTER),
    (dict(ws=WS + 8), hta.ERR_MISALIGNED), (dict(n=255), hta.ERR_WORKSPACE_TOO_SMALL),
    (dict(rope=rope(), q=None), hta.ERR_NULL_POINTER), (dict(rope=rope(rot_dim=1)), hta.ERR_INVALID_OPTION),
    (dict(d=dims(T=0), k=None), hta.OK)])
def test_append_refusals(lib, kw, code):
    a = dict(d=dims(), q=heads(), k=heads(4096 * 2), v=heads(4096 * 3), rope=None, c=cache(), pre=4096 * 4,
             start=4096 * 5, qo=heads(4096 * 6), ws=WS, n=256)
    a.update(kw)
    assert lib.longspec_hta_append_paged(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(d=dims(scale=-1.0)), hta.ERR_INVALID_DIMS), (dict(d=dims(scale=math.nan)), hta.ERR_INVALID_DIMS),
    (dict(d=dims(D=256)), hta.ERR_UNSUPPORTED_D), (dict(c=cache(max_blocks=63)), hta.ERR_INVALID_DIMS),
    (dict(c=cache(v_scale=4096)), hta.ERR_INVALID_OPTION), (dict(window=-1), hta.ERR_INVALID_OPTION),
    (dict(q=heads(h=256)), hta.ERR_INVALID_OPTION), (dict(q=None), hta.ERR_NULL_POINTER),
    (dict(out=None), hta.ERR_NULL_POINTER), (dict(lse=4098), hta.ERR_MISALIGNED), (dict(out=4104), hta.ERR_MISALIGNED),
    (dict(ws=None), hta.ERR_NULL_POINTER), (dict(n=100), hta.ERR_WORKSPACE_TOO_SMALL), (dict(d=dims(T=0), q=None), hta.OK)])
def test_chunk_attention_refusals(lib, kw, code):
    a = dict(d=dims(), q=heads(), c=cache(), pre=4096 * 4, start=4096 * 5, window=0, out=4096 * 6, lse=4096 * 7, ws=WS,
             n=WS_BYTES)
    a.update(kw)
    assert lib.longspec_hta_chunk_attention_paged(*a.values(), None) == code


def test_q8_calls_refuse_bf16_caches_and_bad_arguments(lib):
    q8 = cache(k_scale=4096 * 40, v_scale=4096 * 41)
    d = dims(T=10)
    p = [4096 * i for i in range(1, 9)]
    assert lib.longspec_hta_verify_paged_q8(d, p[0], cache(), *p[1:7], WS, WS_BYTES, None) == hta.ERR_INVALID_OPTION
    assert lib.longspec_hta_prefix_attention_paged_q8(d, p[0], cache(), *p[1:4], WS, WS_BYTES, None) == hta.ERR_INVALID_OPTION
    assert lib.longspec_hta_commit_paged_q8(d, cache(), *p[1:6], WS, 256, None) == hta.ERR_INVALID_OPTION
    for i in range(6):
        bad = list(p[1:7])
        bad[i] = None
        assert lib.longspec_hta_verify_paged_q8(d, p[0], q8, *bad, WS, WS_BYTES, None) == hta.ERR_NULL_POINTER
        bad[i] = p[1] + 8
        assert lib.longspec_hta_verify_paged_q8(d, p[0], q8, *bad, WS, WS_BYTES, None) == hta.ERR_MISALIGNED
    assert lib.longspec_hta_verify_paged_q8(dims(T=257), p[0], q8, *p[1:7], WS, WS_BYTES, None) == hta.ERR_T_TOO_LARGE
    assert lib.longspec_hta_commit_paged_q8(dims(T=300), q8, *p[1:6], WS, 256, None) == hta.ERR_T_TOO_LARGE
    assert lib.longspec_hta_commit_paged_q8(d, q8, *p[1:6], WS, 255, None) == hta.ERR_WORKSPACE_TOO_SMALL


def test_binding_refusals():
    """What the binding itself turns away (tensors on the CPU: it gets as far
    as the device check)."""
    q, k = torch.zeros(4, 8, 128, dtype=BF16), torch.zeros(4, 2, 128, dtype=BF16)
    pos, f = torch.zeros(4, dtype=torch.int32), torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA device"):
        hta.qk_norm_rope(q, k, pos, f)
    for bad in (dict(k=k[:3]), dict(k=k[..., :64]), dict(positions=pos[:3]), dict(inv_freq=torch.zeros(65)),
                dict(inv_freq=f[:0]), dict(rope_scale=0.0), dict(q_weight=torch.zeros(64, dtype=BF16)),
                dict(q=q[None]), dict(positions=pos[::2].repeat(2)[::1][:2])):
        a = dict(q=q, k=k, positions=pos, inv_freq=f)
        a.update(bad)
        with pytest.raises(ValueError):
            hta.qk_norm_rope(**a)
    with pytest.raises(TypeError):
        hta.qk_norm_rope(q, k, pos.long(), f)
    kc = torch.zeros(6, 2, 16, 128, dtype=BF16)
    sc = torch.zeros(6, 2, 16, dtype=torch.uint8)
    table, one, start = torch.zeros(1, 6, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    a = dict(k=k, v=k, k_cache=kc, v_cache=kc, block_table=table, prefix_len=one, q_start=start, L_cap=96)
    for bad in (dict(v=k[:3]), dict(k_cache=kc[..., :64]), dict(block_table=table[0]), dict(q_start=start[:1]),
                dict(k_scale=sc), dict(k_cache=kc[:, :1]), dict(v_cache=kc[:3])):
        with pytest.raises(ValueError):
            hta.append_paged(**{**a, **bad})
    with pytest.raises(TypeError):                                    # scales with a bf16 cache
        hta.append_paged(**a, k_scale=sc, v_scale=sc)
    b = dict(q=q, k_cache=kc, v_cache=kc, block_table=table, prefix_len=one, q_start=start, L_cap=96)
    for bad in (dict(q=q[:, :7]), dict(q=q[..., :64]), dict(prefix_len=one[:0]), dict(block_table=table.repeat(2, 1))):
        with pytest.raises(ValueError):
            hta.chunk_attention_paged(**{**b, **bad})
    k8 = kc.to(torch.float8_e4m3fn)
    tq, kt = torch.zeros(1, 8, 5, 128, dtype=BF16), torch.zeros(1, 2, 5, 128, dtype=BF16)
    par = torch.zeros(1, 5, dtype=torch.int32)
    v = dict(q=tq, k_cache=k8, v_cache=k8, block_table=table, prefix_len=one, k_tree=kt, v_tree=kt, parent=par, L_cap=96,
             k_scale=sc, v_scale=sc)
    for bad in (dict(num_splits=2), dict(k_tree=kt[:, :1]), dict(parent=par[:, :4]), dict(v_scale=None),
                dict(k_scale=sc[:3]), dict(prefix_len=start)):
        with pytest.raises(ValueError):
            hta.verify_paged(**{**v, **bad})
    with pytest.raises(ValueError):
        hta.commit_paged(k8, k8, table, one, kt, kt, one.repeat(2), par, L_cap=96, k_scale=sc, v_scale=sc)


def test_plain_codes_are_the_nearest():
    """The 64-bit quantiser against every e4m3 number, and its scale."""
    table = torch.arange(256, dtype=torch.uint8).view(P.F8).double()
    table = table[torch.isfinite(table)]
    g = torch.Generator().manual_seed(0)
    for scale in (1.0, 1e-3, 300.0, 6e4):
        x = (torch.randn(128, generator=g) * scale).to(BF16)
        val, e = P.quantise_row(x)
        unit = 2.0 ** (e - 127)
        most = float(x.double().abs().max())
        assert e == 134 or most <= 448 * unit
        assert e == 16 or most > 448 * unit / 2
        y = (x.double() / unit).clamp(-448, 448)
        assert ((val - y).abs() <= (table[None] - y[:, None]).abs().amin(1) + 1e-12).all()
        assert torch.equal(val, val.float().to(P.F8).double())
    assert P.quantise_row(torch.tensor([0.0] * 8))[1] == 16
    assert P.quantise_row(torch.tensor([1.0, math.inf]))[1] == 255


def test_plain_rotation_and_attention():
    """The plain forms against their own properties: norms kept by a rotation,
    scores depending on the difference of positions alone, weights of one."""
    g = torch.Generator().manual_seed(0)
    x, y = torch.randn(5, 1, 64, generator=g), torch.randn(5, 1, 64, generator=g)
    f = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float()
    pos = torch.tensor([0, 3, 9, 100, 70000])
    for inter in (False, True):
        a, b = P.norm_rope(x, None, pos, f, inter), P.norm_rope(y, None, pos + 5, f, inter)
        assert torch.allclose(a.norm(dim=-1), x.double().norm(dim=-1))
        a2, b2 = P.norm_rope(x, None, pos * 0, f, inter), P.norm_rope(y, None, pos * 0 + 5, f, inter)
        assert torch.allclose((a * b).sum(-1), (a2 * b2).sum(-1), atol=1e-7)
    k = torch.randn(7, 64, generator=g).double()
    out, lse, absv = P.attend(x[0, 0].double(), k, torch.ones(7, 3).double(), 0.1)
    assert torch.allclose(out, torch.ones(3).double()) and torch.allclose(absv, torch.ones(3).double())
    assert math.isclose(lse, float(torch.logsumexp(k @ x[0, 0].double() * 0.1, 0)))
