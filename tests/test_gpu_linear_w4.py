"""Packing of weights in 4 bits, and products with them, on the GPU against the
definition in 64 bits (tests/_w4.py, where the tolerance is derived)."""
import numpy as np
import pytest
import torch

import _w4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, assert_status_ok, dev, host, status_tensor

pytestmark = pytest.mark.gpu
EPS = {torch.bfloat16: 2.0 ** -7, torch.float32: 0.0}


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


class Weights:
    def __init__(self, rng, N, K, spread=True):
        w = rng.normal(size=(N, K)) * (rng.uniform(0.01, 2, (N, 1)) if spread else 1)
        codes, scales, hs = _w4.quantise(w.astype(np.float32))
        # every code and a wide range of scales, subnormal ones and zero among them
        if N * K > 64:
            codes = np.where(rng.random(codes.shape) < 0.5, rng.integers(0, 16, codes.shape), codes).astype(np.uint8)
            scales = np.where(rng.random(scales.shape) < 0.1, rng.integers(0, 127, scales.shape), scales).astype(np.uint8)
        self.ref = _w4.values(codes, scales, hs)
        self.tiles, self.scale = dev(_w4.pack_codes(codes, scales)), dev(hs)
        self.w = moe.Weight4(self.tiles, N, K, self.scale)


def _check(y, ref, dtype):
    want, tol = ref
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol).all(), "worst error / bound %.2f" % np.max(err / tol)


SIZES = [(1, 1, 1), (1, 31, 16), (1, 128, 128), (2, 33, 17), (7, 200, 129), (8, 1000, 500), (9, 130, 2048), (16, 515, 640), (17, 96, 1000), (5, 5000, 384),
         (31, 257, 256), (32, 64, 1100), (33, 300, 130), (64, 129, 512), (65, 1027, 200), (100, 40, 3001), (129, 260, 448), (257, 385, 320), (300, 700, 96),
         (3, 40, 9000), (12, 40, 5000), (40, 40, 9000), (1, 20, 20011), (1500, 130, 72),
         (2001, 5000, 128), (700, 20000, 200), (800, 9001, 75)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products(T, N, K, dtype):
    rng = np.random.default_rng(T * 7 + N + K)
    w = Weights(rng, N, K)
    x = _bf16(rng.normal(size=(T, K)) * rng.uniform(0.1, 3, K))
    y = torch.full((T, N), float("nan"), dtype=dtype, device=DEV)
    moe.moe_linear_w4(x.to(DEV), w.w, y)
    _check(y, _w4.linear(x.double().numpy(), w.ref, out_eps=EPS[dtype]), dtype)


@pytest.mark.parametrize("T,N,K", [(1, 100, 256), (11, 259, 333), (24, 150, 257), (70, 300, 512), (200, 129, 190)])
@pytest.mark.parametrize("aligned", [True, False])
def test_bias_residual_strides(T, N, K, aligned):
    """Rows of x with a stride, NaN behind and between them; rows of y with a stride, whose other numbers stay."""
    rng = np.random.default_rng(T)
    w = Weights(rng, N, K)
    x = _bf16(rng.normal(size=(T, K)))
    ld, off = (-(-K // 8) * 8 + 16, 8) if aligned else (K + 3, 1)
    buf = torch.full((T * ld + 64,), float("nan"), dtype=torch.bfloat16, device=DEV)
    xs = buf[off:off + T * ld].view(T, ld)[:, :K]
    xs.copy_(x)
    bias, y0 = rng.normal(size=N).astype(np.float32), rng.normal(size=(T, N)).astype(np.float32)
    out = torch.full((T, N + 5), 7.0, device=DEV)
    y = out[:, 2:2 + N]
    y.copy_(dev(y0))
    moe.moe_linear_w4(xs, w.w, y, bias=dev(bias), accumulate=True)
    _check(y, _w4.linear(x.double().numpy(), w.ref, bias.astype(np.float64), y0.astype(np.float64)), torch.float32)
    assert (out[:, :2] == 7).all() and (out[:, 2 + N:] == 7).all()
    half = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    moe.moe_linear_w4(xs, w.w, half, bias=dev(bias))
    _check(half, _w4.linear(x.double().numpy(), w.ref, bias.astype(np.float64), out_eps=EPS[torch.bfloat16]), torch.bfloat16)


@pytest.mark.parametrize("T", [1, 12, 40, 150])
def test_without_row_scales(T):
    rng = np.random.default_rng(3)
    N, K = 70, 160
    codes, scales = rng.integers(0, 16, (N, K)).astype(np.uint8), rng.integers(0, 100, (N, K // 16)).astype(np.uint8)
    w = moe.Weight4(dev(_w4.pack_codes(codes, scales)), N, K)
    x = _bf16(rng.normal(size=(T, K)))
    y = torch.empty(T, N, device=DEV)
    moe.moe_linear_w4(x.to(DEV), w, y)
    _check(y, _w4.linear(x.double().numpy(), _w4.values(codes, scales, np.ones(N))), torch.float32)


@pytest.mark.parametrize("T", [3, 13, 50, 140])
def test_exact_sums(T):
    """Whole numbers whose sums fit 24 bits come out exactly, whatever the order."""
    rng = np.random.default_rng(4)
    N, K = 200, 700
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales = np.full((N, -(-K // 16)), 0x40, np.uint8)       # 2
    w = moe.Weight4(dev(_w4.pack_codes(codes, scales)), N, K)
    x = rng.integers(-100, 101, (T, K))
    y = torch.empty(T, N, device=DEV)
    moe.moe_linear_w4(_bf16(x).to(DEV), w, y)
    assert np.array_equal(host(y).astype(np.float64), x @ _w4.values(codes, scales, np.ones(N)).T)


@pytest.mark.parametrize("T", [4, 20, 90])
def test_non_finite_rows_stay_alone(T):
    rng = np.random.default_rng(5)
    w = Weights(rng, 140, 300)
    x = _bf16(rng.normal(size=(T, 300)))
    clean = torch.empty(T, 140, device=DEV)
    moe.moe_linear_w4(x.to(DEV), w.w, clean)
    x[1, 7], x[3, 299] = float("nan"), float("inf")
    y = torch.empty(T, 140, device=DEV)
    moe.moe_linear_w4(x.to(DEV), w.w, y)
    keep = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(y[keep], clean[keep]) and y[1].isnan().all() and not y[3].isfinite().any()


@pytest.mark.parametrize("T", [1, 16, 33, 128])
def test_large_and_small_numbers(T):
    """Sums of the largest bf16 weights' products and of tiny ones keep their digits."""
    rng = np.random.default_rng(6)
    N, K = 64, 256
    for size in (2.0 ** 100, 2.0 ** -100):
        w = Weights(rng, N, K, spread=False)
        x = _bf16(rng.normal(size=(T, K)) * size)
        y = torch.empty(T, N, device=DEV)
        moe.moe_linear_w4(x.to(DEV), w.w, y)
        want, tol = _w4.linear(x.double().numpy(), w.ref)
        assert (np.abs(host(y) - want) <= tol).all()


@pytest.mark.parametrize("T", [2, 16, 48, 130])
def test_same_bits_every_time_and_in_a_graph(T):
    rng = np.random.default_rng(7)
    w = Weights(rng, 333, 1500)
    x = _bf16(rng.normal(size=(T, 1500))).to(DEV)
    y, z = torch.empty(T, 333, device=DEV), torch.empty(T, 333, device=DEV)
    moe.moe_linear_w4(x, w.w, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_linear_w4(x, w.w, z)
    for _ in range(3):
        z.zero_()
        graph.replay()
        assert torch.equal(y, z)
    # two streams at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(T, 333, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o in zip(streams, outs):
            moe.moe_linear_w4(x, w.w, o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], y) and torch.equal(outs[1], y)


@pytest.mark.parametrize("N,K", [(1, 1), (3, 16), (128, 128), (130, 200), (257, 1000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pack(N, K, dtype):
    rng = np.random.default_rng(N + K)
    w = torch.from_numpy((rng.normal(size=(N, K)) * 10.0 ** rng.uniform(-5, 5, (N, 1))).astype(np.float32)).to(dtype)
    if N > 2:
        w[2] = 0
    st = status_tensor()
    out = moe.Weight4.empty(N, K, DEV)
    out.tensors[0].fill_(255)
    moe.moe_w4_pack(w.to(DEV), out, st)
    codes, scales, hs = _w4.quantise(w.float().numpy())
    assert np.array_equal(host(out.tensors[1]), hs)
    assert np.array_equal(host(out.tensors[0]).reshape(-1), _w4.pack_codes(codes, scales))
    assert_status_ok(st)


def test_pack_strided_and_not_finite():
    rng = np.random.default_rng(8)
    w = rng.normal(size=(20, 40)).astype(np.float32)
    w[4, 5], w[4, 39], w[9] = np.nan, -np.inf, 1e-37     # the last row is too small for a scale of its own
    wide = torch.full((20, 55), float("nan"), device=DEV)
    wide[:, 3:43] = dev(w)
    st = status_tensor()
    out = moe.Weight4.empty(20, 40, DEV)
    moe.moe_w4_pack(wide[:, 3:43], out, st)
    codes, scales, hs = _w4.quantise(w)
    assert np.array_equal(host(out.tensors[0]).reshape(-1), _w4.pack_codes(codes, scales)) and np.array_equal(host(out.tensors[1]), hs)
    assert st.tolist() == [1, 4] and hs[9] == 1


def test_pack_then_multiply_at_once():
    """The product that follows a packing on the same stream sees all of it."""
    rng = np.random.default_rng(9)
    N, K, T = 4000, 2048, 4
    x = _bf16(rng.normal(size=(T, K))).to(DEV)
    ws = [torch.randn(N, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(i)) for i in range(2)]
    packed = [moe.Weight4.pack(w) for w in ws]
    want = []
    for p in packed:
        y = torch.empty(T, N, device=DEV)
        torch.cuda.synchronize()
        moe.moe_linear_w4(x, p, y)
        want.append(y)
    one = moe.Weight4.empty(N, K, DEV)
    for i in range(10):
        y = torch.empty(T, N, device=DEV)
        moe.moe_w4_pack(ws[i % 2], one)
        moe.moe_linear_w4(x, one, y)
        assert torch.equal(y, want[i % 2])


def test_binding_refuses():
    w = moe.Weight4.empty(8, 16, DEV)
    x, y = torch.zeros(2, 16, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 8, device=DEV)
    with pytest.raises(moe.MoeError, match="x: expected 2 rows of 16"):
        moe.moe_linear_w4(x[:, :15], w, y)
    with pytest.raises(moe.MoeError, match="x: expected torch.bfloat16"):
        moe.moe_linear_w4(x.float(), w, y)
    with pytest.raises(moe.MoeError, match="y: expected 2 rows of 8"):
        moe.moe_linear_w4(x, w, y[:1])
    with pytest.raises(moe.MoeError, match="only the rows may be strided"):
        moe.moe_linear_w4(x, w, torch.zeros(8, 2, device=DEV).t())
    with pytest.raises(moe.MoeError, match="bias"):
        moe.moe_linear_w4(x, w, y, bias=torch.zeros(7, device=DEV))
    with pytest.raises(moe.MoeError, match="only fp32"):
        moe.moe_linear_w4(x, w, y.bfloat16(), accumulate=True)
    moe.moe_linear_w4(x[:0], w, y[:0])
