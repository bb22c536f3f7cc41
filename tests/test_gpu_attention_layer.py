"""The attention layer and its pages together, as a server runs them."""
import os
import subprocess
import sys

import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV

pytestmark = pytest.mark.gpu
H, NQ, NKV, D = 256, 8, 2, 64


def _layer(max_tokens, window=0):
    g = torch.Generator(device=DEV).manual_seed(3)
    w = lambda *s: (torch.randn(*s, generator=g, device=DEV) * s[-1] ** -0.5).bfloat16()  # noqa: E731
    ones = torch.ones(D, device=DEV)
    return moe.AttentionLayer(w((NQ + 2 * NKV) * D, H), w(H, NQ * D), NQ, NKV, max_tokens, ones, ones,
                              table=moe.rope_table(600, D, device=DEV), window=window)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("window", [0, 70])
def test_a_prompt_in_one_pass_in_chunks_and_token_by_token(window):
    """What the cache holds does not depend on how the tokens came, and neither do the outputs but for
    rounding: the kernels for many, few and single rows see the same cached numbers."""
    n = 130
    x = torch.randn(n, H, device=DEV).bfloat16()
    layer = _layer(n, window)
    outs, caches = [], []
    for cuts in ([n], [100, 4, 1, 25], [1] * n):
        pages = moe.KvPages(1, 5, NKV, D, 1, 256, DEV)
        cache = pages.layer(0)
        y, at = [], 0
        for c in cuts:
            pages.reserve(_i32([c]))
            y.append(layer.forward(x[at:at + c], cache, _i32([0, c]), c).clone())
            at += c
        assert pages.device_status() == (0, 0) and layer.device_status() == (0, 0)
        assert pages.page_table[0].tolist() == [0, 1, 2, -1]
        k, v = (torch.empty(n, NKV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        moe.moe_kv4_read(cache, _i32([0, n]), k, v)
        outs.append(torch.cat(y).float())
        caches.append((k.float(), v.float()))
    for y, (k, v) in zip(outs[1:], caches[1:]):
        # the projection's sums are ordered by its batch size: a bf16 step of q, k or v, and for few numbers a code
        assert ((k - caches[0][0]).norm() / caches[0][0].norm()) < 0.02 and ((v - caches[0][1]).norm() / caches[0][1].norm()) < 0.02
        assert ((y - outs[0]).norm() / outs[0].norm()) < 0.02


def test_forked_sequences_go_their_own_ways():
    """Two forks of a sequence, each with other next tokens, equal two sequences that never shared a page."""
    n, extra = 100, 30
    x = torch.randn(n, H, device=DEV).bfloat16()
    tails = [torch.randn(extra, H, device=DEV).bfloat16() for _ in range(2)]
    layer = _layer(n)

    def serve(share):
        pages = moe.KvPages(1, 8, NKV, D, 2, 256, DEV)
        cache = pages.layer(0)
        if share:
            pages.reserve(_i32([n, 0]))
            layer.forward(x, cache, _i32([0, n, n]), n)
            pages.assign(_i32([0, 0]))
            assert pages.ref.tolist()[:2] == [2, 2]
        else:
            for s in range(2):
                pages.reserve(_i32([n if s == 0 else 0, n if s == 1 else 0]))
                layer.forward(x, cache, _i32([0, n if s == 0 else 0, n]), n)
        ys = []
        for i in range(extra):
            pages.reserve(_i32([1, 1]))
            ys.append(layer.forward(torch.stack([t[i] for t in tails]), cache, _i32([0, 1, 2]), 1).clone())
        if share:
            assert pages.ref.tolist()[:1] == [2] and int((pages.ref == 1).sum()) == 4
            pages.compact()
            ys.append(layer.forward(torch.stack([t[-1] for t in tails]), cache, _i32([0, 1, 2]), 1).clone())
        else:
            ys.append(layer.forward(torch.stack([t[-1] for t in tails]), cache, _i32([0, 1, 2]), 1).clone())
        assert pages.device_status() == (0, 0)
        return torch.stack(ys)

    assert torch.equal(serve(True), serve(False))


def test_padded_rows_and_a_batch_too_large():
    layer = _layer(4)
    pages = moe.KvPages(1, 4, NKV, D, 3, 128, DEV)
    pages.reserve(_i32([5, 0, 1]))
    y = layer.forward(torch.randn(3, H, device=DEV).bfloat16(), pages.layer(0), _i32([0, 1, 2, 3]), 1)
    assert (y[1] == 0).all() and torch.isfinite(y).all() and layer.device_status() == (0, 0)
    with pytest.raises(moe.MoeError, match="max_tokens"):
        layer.forward(torch.randn(5, H, device=DEV).bfloat16(), pages.layer(0), _i32([0, 1, 2, 3]), 1)


def test_axes_of_pairs():
    assert moe.rope_axes([2, 3, 3], device="cpu").tolist() == [0, 0, 1, 1, 1, 2, 2, 2]
    assert moe.rope_axes([2, 3, 3], True, device="cpu").tolist() == [0, 1, 2, 0, 1, 2, 1, 2]


def test_the_example_runs():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "decode_kv4.py"), "--layers", "2", "--batch", "8", "--prompt", "70",
                        "--steps", "4", "--hidden", "256", "--experts", "16", "--intermediate", "128"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "after forking and packing" in r.stdout
