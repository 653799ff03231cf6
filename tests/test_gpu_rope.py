"""Rotary positions against 64 bits.

Bound of an output, from the formats: its rounding u |out| (2^-11 FP16, 2^-8 BF16; and half a
step of FP16's subnormals, 2^-25), and (|a| + |b|) |gain| 2^-21 for FP32: an angle as a signed
fraction of a half turn is rounded by 2^-25 and cut by 2^-32, that is 2^-23 of a radian, a sine
is good to 2^-23, the gain and the two products round by 2^-24 each.
"""
import math

import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def normal(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def check(x, got, positions, r, inverse=False):
    turns = [math.fmod(f / (2 * math.pi), 1.0) for f in r.freqs]
    # angles without their whole turns, in integers: a position times a fraction of 2^64
    whole = [int(t * 2 ** 64) for t in turns]
    rows = []
    for n in positions.tolist():
        rows.append([((n * w + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2 ** 64 * 2 * math.pi for w in whole])
    w = torch.tensor(rows, dtype=torch.float64, device="cuda").view(len(positions), -1)[:, None, :]
    cos, sin = torch.cos(w) * r.gain, torch.sin(w) * r.gain * (-1 if inverse else 1)
    R = r.rotary
    y = x.double()
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if r.interleaved else (y[..., :R // 2], y[..., R // 2:R])
    g = got.double()
    ga, gb = (g[..., 0:R:2], g[..., 1:R:2]) if r.interleaved else (g[..., :R // 2], g[..., R // 2:R])
    rest = (a.abs() + b.abs()) * abs(r.gain) * 2.0 ** -21 + 2.0 ** -25
    for have, want in ((ga, a * cos - b * sin), (gb, b * cos + a * sin)):
        d = (have - want).abs()
        assert bool((d <= U[x.dtype] * want.abs() + rest).all()), float(d.max())
    assert torch.equal(got[..., R:], x[..., R:])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dim,rotary,heads,kv,rows,kw", [
    (256, None, 6, 2, 33, {}), (256, 64, 24, 4, 5, dict(scaling="yarn", factor=4.0)), (128, 16, 1, 1, 1, {}),
    (128, 80, 5, 0, 17, dict(scaling="linear", factor=8.0)), (128, 128, 16, 1, 130, dict(scaling="ntk", factor=3.0)),
    (48, 48, 3, 3, 9, dict(gain=-0.5)), (72, 32, 7, 2, 2, dict(base=5e5)), (2056, 2048, 1, 1, 3, {}), (16, 16, 40, 8, 64, {})])
def test_rope(dtype, pairs, dim, rotary, heads, kv, rows, kw):
    r = tfx.Rope(dim, rotary, interleaved=pairs, **kw)
    q = normal((rows, heads, dim), dtype, 1)
    k = normal((rows, kv, dim), dtype, 2) if kv else None
    g = torch.Generator().manual_seed(3)
    at = torch.randint(-100, 1 << 20, (rows,), generator=g).int()
    at[:1], at[-1:] = 2 ** 31 - 1, 0
    for inverse in (False, True):
        qo, ko = tfx.rope(r, q, k, at.cuda(), inverse=inverse)
        check(q, qo, at, r, inverse)
        if kv:
            check(k, ko, at, r, inverse)
        else:
            assert ko is None


def test_in_place_in_slices_of_one_buffer():
    """The rotated slices of a q/k/v buffer are the plain call's, everything else stays."""
    dim, hq, hkv, rows = 128, 6, 2, 37
    x = normal((rows + 2, (hq + 2 * hkv) * dim + 8), BF16, 1)
    was = x.clone()
    q = x[1:-1, :hq * dim].unflatten(1, (hq, dim))
    k = x[1:-1, hq * dim:(hq + hkv) * dim].unflatten(1, (hkv, dim))
    at = torch.arange(1000, 1000 + rows, dtype=torch.int32, device="cuda")
    for rotary, pairs in ((32, False), (128, True)):
        r = tfx.Rope(dim, rotary, interleaved=pairs)
        x.copy_(was)
        wq, wk = tfx.rope(r, q, k, at)
        assert torch.equal(x, was)
        tfx.rope(r, q, k, at, out=(q, k))
        assert torch.equal(q, wq) and torch.equal(k, wk)
        was_rest = was.clone()
        was_rest[1:-1, :hq * dim], was_rest[1:-1, hq * dim:(hq + hkv) * dim] = wq.flatten(1), wk.flatten(1)
        assert torch.equal(x, was_rest)


def test_gradient():
    """inverse is the transpose: <g, rope(x)> and <rope(g, inverse), x> agree, and with differences of the formula in 64 bits."""
    r = tfx.Rope(64, 32, scaling="yarn", factor=16.0)
    x, g = normal((11, 3, 64), F16, 1), normal((11, 3, 64), F16, 2)
    at = torch.arange(5000, 5011, dtype=torch.int32, device="cuda")
    y, _ = tfx.rope(r, x, None, at)
    back, _ = tfx.rope(r, g, None, at, inverse=True)
    # sums of 2,112 products whose factors are each off by 2^-11 of themselves at most, and 2^-21 of their pair
    size = float((g.double().abs() * y.double().abs()).sum() + (back.double().abs() * x.double().abs()).sum())
    assert abs(float((g.double() * y.double()).sum() - (back.double() * x.double()).sum())) <= size * (2.0 ** -11 + 2.0 ** -19)
    step = torch.zeros_like(x)
    step[4, 1, 3] = 0.5
    more, _ = tfx.rope(r, x + step, None, at)
    h = float((x + step)[4, 1, 3].double() - x[4, 1, 3].double())
    slope = float((g.double() * (more.double() - y.double())).sum() / h)
    near = float((g.double().abs()[4, 1] * (y.double().abs() + more.double().abs())[4, 1]).sum()) * 2.0 ** -10 / abs(h)
    assert abs(slope - float(back[4, 1, 3])) <= near + 2.0 ** -10


def test_no_rows_and_a_graph():
    r = tfx.Rope(128)
    q = normal((0, 4, 128), F16, 1)
    qo, ko = tfx.rope(r, q, q, torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert qo.shape == q.shape and ko.shape == q.shape
    q, at = normal((8, 4, 128), F16, 2), torch.arange(8, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    tfx.rope(r, q, None, at, out=(out, None))
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        tfx.rope(r, q, None, at, out=(out, None))
    at.add_(77)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    check(q, out, at.cpu(), r)
