"""examples/serve_attention.py over a cache of 8-bit codes: every step's attention against 64 bits over
what the cache holds, and rotated keys in it within half a step of their block's scale."""
import os
import sys

import pytest
import torch

from q8_reference import TOP, assert_near, attend

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("store", [torch.int8, torch.float8_e4m3fn])
def test_serve(store):
    import exl3_trellis_quantized_rot_gb300 as tfx
    import serve_attention as ex
    layer, told = ex.serve(system=300, chats=8, steps=3, page_size=32, store=store)
    c = layer.cache
    assert c.status() == 0 and tfx.attn_error() == 0
    lens = c.lens.tolist()
    assert lens == [300] + [0 if s % 2 else 306 for s in range(1, 9)]
    group, scale = ex.HEADS // ex.KV_HEADS, ex.DIM ** -0.5
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def kv(slot, n):
        return tfx.cache_read(c, 0, ints(slot), ints(0), ints(0, n), n)

    # the system prompt's keys: quantised once, as they were rotated
    x = torch.randn((300, ex.HIDDEN), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").half()
    _, k, _ = tfx.group(layer.qkv, x)
    k = k.unflatten(1, (ex.KV_HEADS, ex.DIM))
    k, _ = tfx.rope(layer.rope, k, None, torch.arange(300, dtype=torch.int32, device="cuda"))
    got, _ = kv(0, 300)
    used = c.tables[0, :-(-300 // 32)].long()
    s = c.k_scale[0][used].reshape(-1, ex.KV_HEADS).repeat_interleave(16, 0)[:300, :, None]
    half = s / 2 if store == torch.int8 else torch.maximum(k.float().abs() * 2 ** -4, s * 2 ** -10)
    assert bool(((got.float() - k.float()).abs() <= half * (1 + 2 ** -9)).all())

    # the last step's rows over what the cache holds now: nothing came after it
    kind, (q, a, y), live = told[-1]
    assert kind == "step" and live == [2, 4, 6, 8]
    assert torch.equal(y, tfx.linear(layer.o, a.flatten(1)))
    most = TOP[store] * float(max(c.v_scale[0][c.tables[s].long().clamp(min=0)].max() for s in live))
    for i, slot in enumerate(live):
        k, v = kv(slot, lens[slot])
        for h in range(ex.HEADS):
            o, A, qk = attend(q[i:i + 1, h], k[:, h // group], v[:, h // group], scale)
            assert_near(a[i:i + 1, h], o, A, qk, lens[slot], ex.DIM, most)
