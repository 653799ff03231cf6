"""examples/serve_attention.py end to end: attention of every step against 64 bits
over what the cache holds (bound: attention_reference), the books at the end."""
import os
import sys

import pytest
import torch

from attention_reference import assert_near, attend

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import __graft_entry__
    __graft_entry__.build_library()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_serve_attention():
    import exl3_trellis_quantized_rot_gb300 as tfx
    import serve_attention as ex
    layer, told = ex.serve(system=300, chats=8, steps=3, page_size=32)
    c = layer.cache
    assert c.status() == 0
    lens = c.lens.tolist()
    assert lens == [300] + [0 if s % 2 else 306 for s in range(1, 9)]
    used = sorted({p for row in c.tables.tolist() for p in row if p >= 0})
    assert used == list(range(len(used))) and int((c.refs > 0).sum()) == len(used)
    # 9 full pages of 32 are shared by the prompt and the four chats that are left
    assert sorted(c.refs.tolist(), reverse=True)[:10] == [5] * 9 + [1]

    group, scale = ex.HEADS // ex.KV_HEADS, ex.DIM ** -0.5

    def kv(slot, n):
        at = c.tables[slot, :-(-n // 32)].long()
        return (x[0, at].reshape(-1, ex.KV_HEADS, ex.DIM)[:n] for x in (c.k, c.v))

    def check(out, q, k, v, seen):
        for h in range(ex.HEADS):
            kh, vh = k[:, h // group], v[:, h // group]
            o, A, qk = attend(q[:, h], kh, vh, seen, scale)
            assert_near(out[:, h], o, A, qk, kh.shape[0], ex.DIM, torch.float16, float(vh.abs().max()))

    _, (q, a, y), _ = told[0]
    k, v = kv(0, 300)
    check(a, q, k, v, torch.ones(300, 300, dtype=torch.bool, device="cuda").tril())
    steps = {}
    for kind, (q, a, y), live in told:
        assert torch.equal(y, tfx.linear(layer.o, a.flatten(1)))
        if kind == "prompt":
            continue
        for i, slot in enumerate(live):
            n = 301 + steps.setdefault(slot, 0)
            steps[slot] += 1
            if slot % 2:  # these have left the cache
                continue
            k, v = kv(slot, n)
            check(a[i:i + 1], q[i:i + 1], k, v, torch.ones(1, n, dtype=torch.bool, device="cuda"))
