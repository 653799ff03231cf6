"""Caches of 8-bit codes that hold values near the end of their rows' type. The nearest code of such
a value can stand for more than the type holds (FP16's largest, 65,504, is 63.97 steps of 1,024 and becomes
64 of them); what is read is the type's largest then, and stays finite."""
import numpy as np
import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx
from q8_reference import BLOCK, TOP, Coded, assert_near, attend

pytestmark = pytest.mark.gpu
F16, BF16, I8, E4M3 = torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(store, act, heads, dim, hq, page=32, pages=12, slots=3, width=6):
    shape = (1, pages, page, heads, dim)
    k, v = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(store) for _ in range(2))
    c = tfx.Cache(k, v, slots, width, act=act)
    tfx.cache_reserve(c, slots, hq)
    return c


def near_the_end(tokens, heads, dim, act, seed):
    """Values from a quarter of the type's largest up to it, of both signs, a fifth of them the largest itself."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.rand((tokens, heads, dim), generator=g, device="cuda") * 0.75 + 0.25
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.2] = 1.0
    sign = torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    return (x.double() * sign * torch.finfo(act).max).to(act)


def saturated(values, act):
    top = torch.finfo(act).max
    return torch.from_numpy(np.clip(values, -top, top)).to(act)


@pytest.mark.parametrize("store", [I8, E4M3])
@pytest.mark.parametrize("act,heads,dim", [(F16, 2, 256), (BF16, 2, 256), (F16, 3, 128), (BF16, 1, 128)])
def test_rows_near_the_end_of_their_type_are_read_back_finite(store, act, heads, dim):
    c = make(store, act, heads, dim, heads)
    n = 53
    k, v = (near_the_end(n, heads, dim, act, seed) for seed in (1, 2))
    assert bool(k.isfinite().all()) and bool(v.isfinite().all())
    v[20, 0, 3] = float("nan")  # one block of one head: NaN as before
    tfx.cache_extend(c, dev(1), dev(0, n))
    tfx.cache_append(c, 0, k, v)
    rk, rv = tfx.cache_read(c, 0, dev(1), dev(0), dev(0, n), n)
    for x, got in ((k, rk), (v, rv)):
        model = Coded(store, heads, dim)
        model.append(x.double().cpu().numpy())
        values = model.values()
        bad = torch.from_numpy(np.broadcast_to(np.isnan(np.repeat(model.scales, BLOCK, 0)[:n, :, None]), values.shape).copy())
        assert bool((torch.from_numpy(values).abs() > torch.finfo(act).max).any())  # there is something to saturate
        assert bool(got.cpu()[bad].isnan().all())
        assert torch.equal(got.cpu()[~bad], saturated(values, act)[~bad])
    # rows that leave the cache and come back are what they were
    tfx.cache_extend(c, dev(0), dev(0, n))
    tfx.cache_append(c, 0, rk, rk)
    assert bool(c.k_scale[0, c.tables[0, :2].long()].isfinite().all())
    back, _ = tfx.cache_read(c, 0, dev(0), dev(0), dev(0, n), n)
    assert torch.equal(back, rk) and c.status() == 0


@pytest.mark.parametrize("store", [I8, E4M3])
@pytest.mark.parametrize("hq,heads,dim", [(6, 2, 256), (4, 4, 128), (20, 1, 128)])
def test_attention_over_values_near_the_end_of_fp16(store, hq, heads, dim):
    """A mean of finite values is finite: beyond FP16's range it is its largest. The bound is that of an unlimited
    result, since a limit brings no two numbers further apart."""
    c = make(store, F16, heads, dim, hq)
    lens = [1, 53, 40]
    at = [0, 1, 54, 94]
    k = near_the_end(94, heads, dim, F16, 1) * 2.0 ** -15
    v = near_the_end(94, heads, dim, F16, 2)
    v[54:] = torch.finfo(F16).max  # the third sequence: all of them the largest
    v[54:, :, ::2] *= -1
    tfx.cache_extend(c, dev(0, 1, 2), dev(*at))
    tfx.cache_append(c, 0, k, v)
    q = torch.randn((3, hq, dim), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(F16)
    got = tfx.attn_decode(c, 0, q, dev(0, 1, 2))
    beyond = False
    for i, n in enumerate(lens):
        kk, vv = (Coded(store, heads, dim) for _ in range(2))
        for m, x in ((kk, k), (vv, v)):
            m.append(x[at[i]:at[i + 1]].double().cpu().numpy())
        most = TOP[store] * float(vv.scales.max())
        kk, vv = (torch.from_numpy(m.values()).cuda() for m in (kk, vv))
        for h in range(heads):
            rows = slice(h * (hq // heads), (h + 1) * (hq // heads))
            out, A, qk = attend(q[i, rows], kk[:, h], vv[:, h], dim ** -0.5)
            beyond = beyond or bool((out.abs() >= 65520).any())
            assert_near(got[i, rows], out.clamp(-65504, 65504), A, qk, n, dim, most)
    assert beyond
    assert bool((got[2].abs() == 65504).all())
    v[70, 0, 5] = float("nan")
    tfx.cache_append(c, 0, k, v)
    got = tfx.attn_decode(c, 0, q, dev(0, 1, 2))
    group = hq // heads
    assert bool(got[2, :group].isnan().all()) and bool(got[2, group:].isfinite().all()) and bool(got[:2].isfinite().all())
