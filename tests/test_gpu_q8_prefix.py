"""The kernel that reads a batch's shared prefix of 8-bit codes once, and only it: that calls above the
limit of 64 MiB (batch * shared tokens) reach it is told by their number of launches. Scores and values
that rise and fall along the prefix by less and by more than what moves its references, shares of many
tiles, more tiles of rows than SMs, and steps one behind another."""
import math
import os
import subprocess
import sys

import pytest
import torch

import exl3_trellis_quantized_rot_gb300 as tfx
from q8_reference import BLOCK, TOP, assert_near
from test_gpu_q8_large import behind, check, dev, make, normal, values

pytestmark = pytest.mark.gpu
F16, BF16, I8, E4M3 = torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def decode(*args, launches=3, **kw):
    """attn_decode, which is the prefix's kernel, the own tokens' and the join, or the last two."""
    n = tfx.launch_count()
    out = tfx.attn_decode(*args, **kw)
    assert tfx.launch_count() - n == launches
    assert tfx.attn_error() == 0
    return out


# 130 sequences of 32 heads over 2,048 tokens: 33 tiles of rows, so that a share has 8 tiles of 64 keys (on
# 152 SMs) and its references go on from tile to tile. Scores rise from a block of 16 keys to the next by 2^rise
# and values by 2^grow, 32 blocks long, then again.
@pytest.mark.parametrize("store", [I8, E4M3])
@pytest.mark.parametrize("act,dim", [(F16, 128), (BF16, 256)])
@pytest.mark.parametrize("rise,grow", [(7.9, 0), (8.2, 0), (1.9, 0), (2.1, 0), (0.1, 0.1), (-2.0, 0.3), (0.0, 0.3), (0.0, -0.3),
                                       (-4.0, 3.5), (4.0, -3.5), (3.0, 0.9)])
def test_scores_and_values_that_rise_along_a_prefix(store, act, dim, rise, grow):
    n, hq, shared, page = 130, 32, 2048, 64
    if act == F16:
        grow = math.copysign(min(abs(grow), 0.4), grow)  # 2^13 in all
    c = make(store, act, shared // page + 1, page, 1, dim, n + 1, shared // page, n, hq)
    b = torch.arange(shared, device="cuda") // BLOCK % 32 - 16
    k, v = normal((shared, 1, dim), act, 1, 0.05), normal((shared, 1, dim), F16, 2).float()
    k[:, 0, 0] = (b * rise * math.log(2)).to(act)
    v = (v * torch.exp2(b * grow)[:, None, None]).to(act)
    tfx.cache_extend(c, dev([n]), dev([0, shared]))
    tfx.cache_append(c, 0, k, v)
    tfx.cache_fork(c, dev([n] * n), dev(range(n)))
    assert c.status() == 0
    q = normal((n, hq, dim), act, 3, 0.1)
    q[:, :, 0] = torch.tensor([1.0, -1.0, 0.5, 0.0], device="cuda")[torch.arange(hq, device="cuda") % 4].to(act)
    got = decode(c, 0, q, dev(range(n)), shared=shared, scale=1.0)
    kk, vv = (x[:, 0] for x in values(c, n, shared))
    scales = c.v_scale[0][c.tables[n, :shared // page].long()].double().reshape(-1)
    # the test reaches what it is for: V's scales differ by as much as they should
    assert float(scales.max() / scales.min()) >= 2.0 ** (abs(grow) * 31 - 2)
    rows = q.double().flatten(0, 1)
    p = torch.softmax(rows @ kk.T, 1)
    # of each row: its sum of |q k|, and the largest product of a probability and a block's scale of V, of which the
    # weights' FP16 steps are
    qk = (rows.abs() @ kk.abs().T).amax(1, keepdim=True)
    most = TOP[store] * (p.view(len(rows), -1, BLOCK).amax(2) * scales).amax(1, keepdim=True)
    assert_near(got.flatten(0, 1), p @ vv, p @ vv.abs(), qk, shared, dim, most, float(vv.abs().max()))


SHAPES = [
    (BF16, 24, 4, 256, 64, 1605, 30), (F16, 8, 1, 128, 16, 703, 400), (F16, 128, 1, 256, 32, 320, 430), (BF16, 6, 2, 128, 128, 5000, 64),
    (F16, 16, 16, 128, 16, 300, 60), (BF16, 20, 1, 256, 16, 256, 530), (F16, 12, 2, 256, 64, 575, 130), (BF16, 7, 7, 256, 16, 4703, 4)]


@pytest.mark.parametrize("store", [I8, E4M3])
@pytest.mark.parametrize("act,hq,hkv,dim,page,shared,n", SHAPES)
def test_shapes_that_reach_the_kernel(store, act, hq, hkv, dim, page, shared, n):
    """Tiles of rows whole and partly filled, more of them than SMs, one share and many, one tile a share and many."""
    width = shared // page + 3
    c = make(store, act, width + 4 * n, page, hkv, dim, n + 4, width, n + 3, hq)
    behind(c, n, shared, n, lambda i: 1 + i % 19, (100, 17))
    order = list(range(n)) + [n + 1, n + 2, n + 3]
    q = normal((n + 3, hq, dim), act, 7, 0.3)
    got = decode(c, 0, q, dev(order), shared=shared)
    check(c, q, order, got, shared, n, dim ** -0.5)
    assert torch.equal(decode(c, 0, q, dev(order), shared=shared), got)
    decode(c, 0, q[:2], dev(order[:2]), shared=shared, launches=2)
    decode(c, 0, q, dev(order), launches=2)


@pytest.mark.parametrize("store", [I8, E4M3])
def test_steps_behind_a_prefix_one_after_another(store):
    """Rotation, extend, append and attention behind a prefix, launch upon launch, in a graph and with dependent launches
    off: the same bits."""
    n, shared, page, hq, hkv, dim, act = 40, 1005, 16, 24, 4, 256, BF16
    r = tfx.Rope(dim, 64)

    def cache():
        c = make(store, act, shared // page + 2 + 4 * n, page, hkv, dim, n + 1, shared // page + 4, n, hq)
        behind(c, n, shared, n, lambda i: 1 + i % 19)
        return c

    a, b, warm = cache(), cache(), cache()
    seqs, at = dev(range(n)), dev(range(n + 1))
    x = {name: normal((n, h, dim), act, 9 + h) for name, h in (("q", hq), ("k", hkv), ("v", hkv))}
    rotated = [(torch.empty_like(x["q"]), torch.empty_like(x["k"])) for _ in range(3)]
    out = [torch.empty_like(x["q"]) for _ in range(3)]

    def step(c, i):
        tfx.cache_extend(c, seqs, at)
        q, k = tfx.rope(r, x["q"], x["k"], (c.lens[:n] - 1).contiguous(), out=rotated[i])
        tfx.cache_append(c, 0, k, x["v"])
        launched = tfx.launch_count()
        tfx.attn_decode(c, 0, q, seqs, shared=shared, out=out[i])
        assert tfx.launch_count() - launched == 3

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm, 2)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(b, 1)
            step(b, 1)
    for _ in range(6):
        x["q"].neg_().mul_(1.125)
        x["k"].mul_(1.25)
        x["v"].neg_().mul_(1.5)
        torch.cuda.synchronize()
        old = tfx.set_pdl(0)
        try:
            step(a, 0)
            step(a, 0)
        finally:
            tfx.set_pdl(old)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.book, b.book) and torch.equal(out[0], out[1])
        for u, v in ((a.k, b.k), (a.v, b.v)):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
        for u, v in ((a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
            assert torch.equal(u.nan_to_num(), v.nan_to_num())
    assert a.status() == 0 and b.status() == 0 and tfx.attn_error() == 0


@pytest.mark.parametrize("store", [I8, E4M3])
@pytest.mark.parametrize("hq,hkv,dim,page,shared,n", [(24, 4, 256, 16, 1211, 30), (6, 2, 128, 64, 100, 5)])
def test_layers_have_their_own_codes_and_scales(store, hq, hkv, dim, page, shared, n):
    """Attention, with and without the prefix's kernel, and reads of three layers that hold different values."""
    layers, act = 3, F16
    width = shared // page + 3
    c = make(store, act, width + 3 * n, page, hkv, dim, n + 1, width, n, hq, layers=layers)

    def put(adds, seed):
        at = [0]
        for _, m in adds:
            at.append(at[-1] + m)
        tfx.cache_extend(c, dev(s for s, _ in adds), dev(at))
        for layer in range(layers):
            tfx.cache_append(c, layer, *(normal((at[-1], hkv, dim), act, seed + 10 * layer + i, 4.0 ** layer) for i in range(2)))

    put([(n, shared)], 1)
    tfx.cache_fork(c, dev([n] * n), dev(range(n)))
    put([(i, 1 + i % 5) for i in range(n)], 3)
    assert c.status() == 0
    q = normal((n, hq, dim), act, 7, 0.05)
    launches = 3 if n * (shared // BLOCK * BLOCK) * hkv * dim * 2 > 64 << 20 else 2
    outs = [decode(c, layer, q, dev(range(n)), shared=shared, launches=launches) for layer in range(layers)]
    for layer, got in enumerate(outs):
        # the same cache as one of a single layer
        one = tfx.Cache(*(x[layer:layer + 1].contiguous() for x in (c.k, c.v)), n + 1, width, book=c.book.clone(),
                        k_scale=c.k_scale[layer:layer + 1].contiguous(), v_scale=c.v_scale[layer:layer + 1].contiguous(), act=act)
        tfx.cache_reserve(one, n, hq)
        check(one, q, list(range(n)), got, shared, n, dim ** -0.5)
        lists = dev([n, 0]), dev([3, 0]), dev([0, shared - 3, shared - 3 + 7])
        for u, v in zip(tfx.cache_read(c, layer, *lists, shared + 4), tfx.cache_read(one, 0, *lists, shared + 4)):
            assert torch.equal(u, v)
        assert one.status() == 0


FIRST = """
import torch
import exl3_trellis_quantized_rot_gb300 as tfx
h = lambda *s: torch.randn(s, device="cuda").half()
i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
pages = lambda: torch.empty((1, 80, 16, 1, 256), dtype=torch.int8, device="cuda")
c = tfx.Cache(pages(), pages(), 4, 70, act=torch.float16)
tfx.cache_reserve(c, 140, 8)
r = tfx.Rope(256, 64)
k, kr, q, out, rk, rv = h(1000, 1, 256), h(1000, 1, 256), h(140, 8, 256), h(140, 8, 256), h(1000, 1, 256), h(1000, 1, 256)
s, d, o, same, z = i(0), i(1), i(0, 1000), i(*[0] * 140), i(0)
at = torch.arange(1000, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    tfx.rope(r, k, None, at, out=(kr, None))
    tfx.cache_extend(c, s, o)
    tfx.cache_append(c, 0, kr, k)
    tfx.attn_decode(c, 0, q, same, shared=1000, out=out)  # the prefix's kernel, the own tokens', the join
    tfx.attn_decode(c, 0, q, same, out=q)
    tfx.cache_read(c, 0, s, z, o, 1000, out=(rk, rv))
    tfx.cache_fork(c, s, d)
g.replay()
torch.cuda.synchronize()
assert c.lens.tolist() == [1000, 1000, 0, 0] and c.status() == 0 and tfx.attn_error() == 0
assert torch.equal(kr, tfx.rope(r, k, None, at)[0])
read = tfx.cache_read(c, 0, s, z, o, 1000)
assert torch.equal(read[0], rk) and torch.equal(read[1], rv)
# two ways over the same codes: apart by the bounds of each, 2^-10 of the largest value and the output's two steps
assert float((out.float() - q.float()).abs().max()) <= float(rv.float().abs().max()) * 2.0 ** -8
"""


def test_first_calls_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST], check=True, cwd=root, timeout=300)


def test_calls_of_several_streams_at_once():
    """Two caches and a prompt on three streams, kernels of each with tensor memory of their own: the bits of one after another."""
    shapes = [(I8, F16, 8, 1, 128, 16, 703, 400), (E4M3, BF16, 24, 4, 256, 64, 1605, 30)]
    calls = []
    for store, act, hq, hkv, dim, page, shared, n in shapes:
        width = shared // page + 3
        c = make(store, act, width + 4 * n, page, hkv, dim, n + 1, width, n, hq)
        behind(c, n, shared, n, lambda i: 1 + i % 19)
        q, seqs, out = normal((n, hq, dim), act, 7, 0.3), dev(range(n)), normal((n, hq, dim), act, 8)
        calls.append((lambda c=c, q=q, seqs=seqs, shared=shared, out=out: tfx.attn_decode(c, 0, q, seqs, shared=shared, out=out), out))
    q, k, out = normal((3000, 24, 128), F16, 1), normal((3000, 4, 128), F16, 2), normal((3000, 24, 128), F16, 3)
    off = torch.tensor([0, 1700, 3000], dtype=torch.int32)
    calls.append((lambda: tfx.attn_prompt(q, k, k, off, out=out), out))
    want = [call().clone() for call, _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for _, out in calls:
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for s, (call, _) in zip(streams, calls):
                with torch.cuda.stream(s):
                    call()
        torch.cuda.synchronize()
        for w, (_, out) in zip(want, calls):
            assert torch.equal(out, w)
    assert tfx.attn_error() == 0
