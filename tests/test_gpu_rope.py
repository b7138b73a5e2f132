"""GPU tests of the per-head norm and rotation, against the definition in 64 bits.

Tolerances, per value, before any run: the kernel works in fp32.  The mean square of d values is
off by at most d * 2^-24 of itself, its root by half of that: d/2 * 2^-24 <= 2^-18; the products
with the weight, cosine and sine add a few 2^-24, the angle (a turn's fraction rounded to fp32)
at most 2 pi * 2^-25 and sincospi two steps: together under 2^-17 of the pair's length.  The one
rounding to bf16 adds 2^-8 of the value.
"""

import math

import pytest
import torch

from block_sparse_attention_gather_b200 import (SparkError, spark_attend_dense, spark_qk_norm_rope,
                                                spark_rope_frequencies)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def reference(x, w, eps, pos, freq, axes, interleaved, scale):
    """(y, length of the value's pair) in 64 bits."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    size = y.abs().clone()
    if pos is None:
        return y, size
    n = freq.numel()
    axis = torch.repeat_interleave(torch.arange(len(axes)), torch.tensor(axes)).to(DEV)
    t = pos.double()[:, axis] * freq.double()
    c, s = torch.cos(t) * scale, torch.sin(t) * scale
    ia = torch.arange(n, device=DEV) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else n)
    a, b = y[..., ia], y[..., ib]
    out = y.clone()
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = torch.hypot(a, b) * scale
    return out, size


def check(got, want):
    y, size = want
    tol = 2.0 ** -17 * size + 1e-30
    if got.dtype == BF:
        tol = tol + 2.0 ** -8 * y.abs()
    worst = ((got.double() - y).abs() / tol).max().item()
    assert worst <= 1.0, f"off by {worst:.2f} of the tolerance"


def inputs(seed, H, N, d, dtype, packed=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if packed:
        x = (torch.randn(N, 3, H, d, generator=g, device=DEV) * 2).to(dtype)
        return [x[:, i].transpose(0, 1) for i in range(3)], g
    return [(torch.randn(H, N, d, generator=g, device=DEV) * 2).to(dtype) for _ in range(3)], g


CASES = [  # H, N, d, axes, far
    (1, 1, 64, [32], 10), (3, 1, 128, [64], 2 ** 31 - 1), (2, 33, 128, [16, 24, 24], 100),
    (24, 5, 64, [8, 12, 12], 60), (5, 130, 128, [20], 1000), (4, 64, 64, [3, 4], 50),
    (2, 100, 128, [1], 9), (1, 1000, 128, [10, 11, 12, 13], 4000), (7, 31, 64, [5, 0, 26], 77),
    (16, 300, 128, [0, 64], 30)]


@pytest.mark.parametrize("H,N,d,axes,far", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_norm_and_rotation(H, N, d, axes, far, interleaved, dtype):
    (Q, K, V), g = inputs(H * N, H, N, d, dtype, packed=N % 2 == 1)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
    pos = torch.randint(-far, far, (N, len(axes)), generator=g, device=DEV, dtype=torch.int64).int()
    freq, _ = spark_rope_frequencies(axes)
    freq = freq.to(DEV)
    got = spark_qk_norm_rope(Q, K, V, wq, wk, 1e-6, pos, freq, axes, interleaved, 1.25)
    check(got[0], reference(Q, wq, 1e-6, pos, freq, axes, interleaved, 1.25))
    check(got[1], reference(K, wk, 1e-6, pos, freq, axes, interleaved, 1.25))
    assert torch.equal(got[2], V.contiguous())
    assert all(t.is_contiguous() for t in got)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("which", ["q", "k", "none"])
def test_parts_left_out(dtype, which):
    (Q, K, V), g = inputs(3, 3, 50, 128, dtype)
    w = 1 + 0.3 * torch.randn(128, generator=g, device=DEV)
    pos = torch.rand(50, generator=g, device=DEV) * 1e5          # fractional, one axis
    freq, _ = spark_rope_frequencies([32])
    freq = freq.to(DEV)
    wq, wk = (w if which == "q" else None), (w if which == "k" else None)
    got = spark_qk_norm_rope(Q, K, None, wq, wk, positions=pos, inv_freq=freq)
    assert got[2] is None
    check(got[0], reference(Q, wq, 1e-6, pos[:, None], freq, [32], False, 1.0))
    check(got[1], reference(K, wk, 1e-6, pos[:, None], freq, [32], False, 1.0))
    only = spark_qk_norm_rope(Q, q_weight=w)                     # no rotation, no keys
    assert only[1] is None and only[2] is None
    check(only[0], reference(Q, w, 1e-6, None, None, None, False, 1.0))
    moved = spark_qk_norm_rope(Q, K, V)                          # the layout change alone
    for a, b in zip(moved, (Q, K, V)):
        assert torch.equal(a, b.contiguous())


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("shift,stride", [(0, 130), (1, 131), (2, 132), (4, 136), (3, 128)])
def test_any_alignment_and_stride(dtype, shift, stride):
    H, N, d = 3, 40, 128
    base = torch.randn(H * N * stride + 64, device=DEV).to(dtype)
    Q = torch.as_strided(base, (H, N, d), (N * stride, stride, 1), shift)
    K = torch.as_strided(base, (H, N, d), (stride, H * stride, 1), shift)
    w = torch.rand(d, device=DEV) + 0.5
    pos = torch.arange(N, device=DEV, dtype=torch.int32)[:, None]
    freq = spark_rope_frequencies([64])[0].to(DEV)
    flat = torch.empty(2, H * N * d + 8, device=DEV, dtype=dtype)
    outs = [flat[i, shift:shift + H * N * d].view(H, N, d) for i in range(2)]
    spark_qk_norm_rope(Q, K, None, w, w, 1e-6, pos, freq, [64], Q_out=outs[0], K_out=outs[1])
    check(outs[0], reference(Q, w, 1e-6, pos, freq, [64], False, 1.0))
    check(outs[1], reference(K, w, 1e-6, pos, freq, [64], False, 1.0))


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_on_another_stream(interleaved):
    (Q, K, V), g = inputs(5, 4, 77, 64, BF, packed=False)
    w = torch.rand(64, generator=g, device=DEV) + 0.5
    pos = torch.arange(77, device=DEV, dtype=torch.int32)[:, None]
    freq = spark_rope_frequencies([32])[0].to(DEV)
    want = spark_qk_norm_rope(Q, K, V, w, w, 1e-6, pos, freq, [32], interleaved)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    spark_qk_norm_rope(Q, K, V, w, w, 1e-6, pos, freq, [32], interleaved, Q_out=Q, K_out=K,
                       V_out=V, stream=side)
    side.synchronize()
    for a, b in zip((Q, K, V), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shift", [0, 2])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_every_count_of_pairs_and_what_lies_behind_them(dtype, interleaved, shift):
    base = torch.randn(9 * 128 + 8, device=DEV).to(dtype)
    pos = torch.tensor([5, -7, 100], device=DEV, dtype=torch.int32)[:, None]
    for pairs in range(1, 65):
        x = base.clone()[shift:shift + 9 * 128].view(3, 3, 128)
        if shift == 0 and pairs < 64:
            x[..., 2 * pairs:] = torch.tensor([float("inf"), float("nan")], device=DEV,
                                              dtype=dtype).repeat(64 - pairs)
        freq = spark_rope_frequencies([pairs])[0].to(DEV)
        got = spark_qk_norm_rope(x, None, None, None, None, 1e-6, pos, freq, [pairs], interleaved)[0]
        assert torch.equal(got[..., 2 * pairs:].nan_to_num(7.0), x[..., 2 * pairs:].nan_to_num(7.0))
        ones = torch.where(torch.isfinite(x), x, torch.ones_like(x))
        want = reference(ones, None, 1e-6, pos, freq, [pairs], interleaved, 1.0)
        check(got[..., :2 * pairs], [t[..., :2 * pairs] for t in want])


@pytest.mark.parametrize("N", [1, 77, 5000])
@pytest.mark.parametrize("captured", [False, True])
def test_calls_that_feed_each_other(N, captured):
    """Each call reads what the one before it wrote and writes what that one read, without a pause;
    the dense attention between them reads the keys and writes the next queries."""
    (Q, K, V), g = inputs(N, 4, N, 128, BF, packed=False)
    w = torch.rand(128, generator=g, device=DEV) + 0.5
    pos = torch.arange(N, device=DEV, dtype=torch.int32)[:, None]
    freq = spark_rope_frequencies([64])[0].to(DEV)

    def chain(pause):
        a, b = [t.clone() for t in (Q, K, V)], [torch.empty_like(t) for t in (Q, K, V)]
        for i in range(6):
            spark_qk_norm_rope(*a, w, w, 1e-6, pos, freq, [64], i % 2 == 1, Q_out=b[0], K_out=b[1],
                               V_out=b[2])
            pause()
            if i % 3 == 2:
                spark_attend_dense(b[0], b[1], b[2], out=a[0])
                pause()
                spark_qk_norm_rope(a[0], b[1], b[2], w, w, 1e-6, pos, freq, [64], K_out=a[1],
                                   Q_out=b[0], V_out=a[2])
                pause()
                b[1], a[1] = a[1], b[1]
                b[2], a[2] = a[2], b[2]
            a, b = b, a
        return a

    want = chain(torch.cuda.synchronize)
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain(lambda: None)
        for _ in range(2):
            graph.replay()
    else:
        got = chain(lambda: None)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.isfinite(x).all() and torch.equal(x, y)


def test_inputs_that_repeat_themselves():
    """Strides of 0: one head shared by all (Q), one token by all (K)."""
    H, N, d = 5, 60, 128
    one = torch.randn(1, N, d, device=DEV).to(BF)
    row = torch.randn(H, 1, d, device=DEV).to(BF)
    w = torch.rand(d, device=DEV) + 0.5
    pos = torch.arange(N, device=DEV, dtype=torch.int32)[:, None]
    freq = spark_rope_frequencies([64])[0].to(DEV)
    q, k, v = spark_qk_norm_rope(one.expand(H, N, d), row.expand(H, N, d), one.expand(H, N, d), w, w,
                                 1e-6, pos, freq, [64], True)
    check(q, reference(one.expand(H, N, d), w, 1e-6, pos, freq, [64], True, 1.0))
    check(k, reference(row.expand(H, N, d), w, 1e-6, pos, freq, [64], True, 1.0))
    assert torch.equal(v, one.expand(H, N, d))


def test_zero_rows_infinities_and_graph_replay():
    (Q, K, V), g = inputs(6, 2, 20, 128, torch.float32, packed=False)
    Q[0, 3] = 0
    Q[1, 4, 5] = math.inf
    w = torch.ones(128, device=DEV)
    got = spark_qk_norm_rope(Q, K, V, w, w)
    assert (got[0][0, 3] == 0).all()
    assert torch.isnan(got[0][1, 4, 5]) and (got[0][1, 4, :5] == 0).all()
    outs = [torch.empty_like(t) for t in got]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spark_qk_norm_rope(Q, K, V, w, w, Q_out=outs[0], K_out=outs[1], V_out=outs[2])
    Q.copy_(K)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], V)


def test_more_elements_than_32_bits():
    H, N, d = 2, 9_000_000, 128                              # 2.3e9 elements, 4.6 GB
    Q = torch.empty(H, N, d, dtype=BF, device=DEV)
    last = torch.randn(H, 50, d, device=DEV).to(BF)
    Q[:, -50:] = last
    w = torch.rand(d, device=DEV) + 0.5
    pos = torch.zeros(N, 1, dtype=torch.int32, device=DEV)
    pos[-50:, 0] = torch.arange(50, device=DEV)
    freq = spark_rope_frequencies([64])[0].to(DEV)
    spark_qk_norm_rope(Q, q_weight=w, positions=pos, inv_freq=freq, Q_out=Q)
    check(Q[:, -50:], reference(last, w, 1e-6, pos[-50:], freq, [64], False, 1.0))


def test_binding_refusals():
    (Q, K, V), g = inputs(9, 2, 6, 64, BF, packed=False)
    w = torch.ones(64, device=DEV)
    pos = torch.zeros(6, 2, dtype=torch.int32, device=DEV)
    f = torch.ones(10, device=DEV)
    good = dict(Q=Q, K=K, V=V, q_weight=w, k_weight=w, positions=pos, inv_freq=f, axis_pairs=[4, 6])
    spark_qk_norm_rope(**good)
    for change in (dict(Q=Q.half()), dict(Q=Q[0]), dict(Q=Q.cpu()), dict(Q=Q.transpose(1, 2)),
                   dict(K=K.float()), dict(K=K[:1]), dict(K=None), dict(V=V[:, :3]), dict(V=[1]),
                   dict(q_weight=w.to(BF)), dict(k_weight=w[:32]), dict(positions=pos.long()),
                   dict(positions=pos[:5]), dict(positions=None), dict(inv_freq=None),
                   dict(inv_freq=f.double()), dict(axis_pairs=[4, 5]), dict(axis_pairs=[10]),
                   dict(axis_pairs=None), dict(Q_out=Q.float()), dict(K_out=K[:, :5].contiguous()),
                   dict(Q_out=V.transpose(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            spark_qk_norm_rope(**{**good, **change})
    for change in (dict(axis_pairs=[-1, 11]), dict(eps=-1.0), dict(Q_out=K), dict(V_out=Q)):
        with pytest.raises(SparkError):
            spark_qk_norm_rope(**{**good, **change})
