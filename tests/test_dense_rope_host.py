"""Norm and rotation, dense attention and key ranges without a GPU: the library refuses bad
arguments on the host, the binding refuses what would not be those arguments, and the rotation
frequencies follow their formulas."""

import ctypes
import math

import pytest
import torch

from block_sparse_attention_gather_b200 import (
    SparkError, lib, spark_attend_dense, spark_attend_dense_workspace_size, spark_attend_ranges,
    spark_bsa_forward_joint, spark_bsa_workspace_size_ctx, spark_bsa_workspace_size_joint,
    spark_qk_norm_rope, spark_rope_frequencies)

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(0x100000)
OUT = ctypes.c_void_p(0x900000)


@pytest.fixture(scope="module")
def L():
    from block_sparse_attention_gather_b200.build import build_library, is_stale
    if is_stale():
        build_library()
    return lib()


def dense(L, **kw):
    a = dict(Q=P, K=P, V=P, Kc=P, Vc=P, H=2, nq=300, nk=1000, nc=10, d=128, ranges=None, out=OUT,
             out_dtype=0, lse=P, ws=P, ws_bytes=0, err=None, stream=None)
    a.update(kw)
    return L.spark_attend_dense(*a.values())


def test_dense_refusals(L):
    assert dense(L, Q=None) == INVALID
    assert dense(L, out=None) == INVALID
    assert dense(L, K=None) == INVALID
    assert dense(L, Vc=None) == INVALID
    assert dense(L, H=0) == INVALID
    assert dense(L, nq=0) == INVALID
    assert dense(L, nk=-1) == INVALID
    assert dense(L, nc=-1) == INVALID
    assert dense(L, d=96) == UNSUPPORTED
    assert dense(L, H=70000) == UNSUPPORTED
    assert dense(L, nk=(1 << 30) + 1) == UNSUPPORTED
    assert dense(L, nc=(1 << 20) + 1) == UNSUPPORTED
    assert dense(L, out_dtype=2) == INVALID
    for name in ("Q", "K", "V", "Kc", "Vc", "out", "ranges"):
        assert dense(L, **{name: ctypes.c_void_p(0x100008)}) == INVALID
    assert dense(L, lse=ctypes.c_void_p(0x100002)) == INVALID
    assert dense(L, ws=None) == WORKSPACE
    assert dense(L, ws_bytes=100) == WORKSPACE
    assert dense(L, ws=ctypes.c_void_p(0x100010), ws_bytes=1 << 40) == WORKSPACE
    assert dense(L, out=P, ws_bytes=1 << 40) == INVALID          # over an input
    # an empty key set needs no pointers: the next check is reached
    assert dense(L, K=None, V=None, nk=0) == WORKSPACE
    assert dense(L, Kc=None, Vc=None, nc=0) == WORKSPACE


def test_dense_workspace_size(L):
    size = spark_attend_dense_workspace_size
    assert size(24, 1, 60480, 0, 128) >= 24 * (128 * 4 + 8)
    assert size(24, 30240, 30240, 0, 128) == 256          # enough rows: nothing is split
    assert size(2, 0, 100, 0, 128) == 0
    assert size(2, 1, 100, 0, 80) == 0
    for nq in (1, 77, 128, 129, 512, 4000, 1 << 20):
        for nk in (0, 1, 1000, 241920, 1 << 24):
            assert 256 <= size(24, nq, nk, 512, 128) <= (1 << 30)


def test_ranges_refusals(L):
    f = L.spark_attend_ranges
    assert f(10, 2, None, P, P, None, 0, P, None, None) == INVALID
    assert f(10, 2, P, P, P, None, 0, None, None, None) == INVALID
    assert f(0, 2, P, P, P, None, 0, P, None, None) == INVALID
    assert f(10, 0, P, P, P, None, 0, P, None, None) == INVALID
    assert f((1 << 30) + 1, 2, P, P, P, None, 0, P, None, None) == UNSUPPORTED
    assert f(10, 2, P, P, P, None, 0, ctypes.c_void_p(0x100008), None, None) == INVALID


def rope(L, **kw):
    a = dict(Q=P, K=P, V=P, dtype=0, H=2, N=10, d=128, strides=None, wq=P, wk=P, eps=1e-6, pos=P,
             f32=0, naxes=1, axis_pairs=(ctypes.c_int32 * 4)(64), pairs=64, freq=P, inter=0,
             scale=1.0, qo=OUT, ko=ctypes.c_void_p(0xa00000),
             vo=ctypes.c_void_p(0xb00000), stream=None)
    a.update(kw)
    return L.spark_qk_norm_rope(*a.values())


def test_rope_refusals(L):
    assert rope(L, Q=None) == INVALID
    assert rope(L, qo=None) == INVALID
    assert rope(L, ko=None) == INVALID
    assert rope(L, vo=None) == INVALID
    assert rope(L, dtype=2) == INVALID
    assert rope(L, H=0) == INVALID
    assert rope(L, N=0) == INVALID
    assert rope(L, d=96) == UNSUPPORTED
    assert rope(L, H=70000) == UNSUPPORTED
    for eps in (-1e-6, math.nan, math.inf):
        assert rope(L, eps=eps) == INVALID
    assert rope(L, scale=math.nan) == INVALID
    assert rope(L, pairs=65) == INVALID
    assert rope(L, pairs=-1) == INVALID
    assert rope(L, pairs=63) == INVALID                          # the axes hold 64
    assert rope(L, pos=None) == INVALID
    assert rope(L, freq=None) == INVALID
    assert rope(L, axis_pairs=None) == INVALID
    assert rope(L, naxes=0) == INVALID
    assert rope(L, naxes=5, axis_pairs=(ctypes.c_int32 * 5)(64)) == UNSUPPORTED
    assert rope(L, naxes=2, axis_pairs=(ctypes.c_int32 * 4)(65, -1)) == INVALID
    assert rope(L, Q=ctypes.c_void_p(0x100001)) == INVALID       # half an element
    # in place needs the output's own layout, and no other tensor's place
    strides = (ctypes.c_int64 * 6)(128, 256, 1280, 128, 1280, 128)
    assert rope(L, qo=P, strides=strides, K=None, wk=None, V=None) == INVALID
    assert rope(L, ko=OUT) == INVALID
    assert rope(L, qo=ctypes.c_void_p(0x200000), K=ctypes.c_void_p(0x200000)) == INVALID


def test_frequencies():
    n, base = 64, 10000.0
    f, scale = spark_rope_frequencies([n], base)
    want = torch.tensor([base ** (-i / n) for i in range(n)], dtype=torch.float64)
    assert scale == 1.0 and torch.equal(f, want.float())
    f, _ = spark_rope_frequencies([16, 0, 24], 500.0)
    want = [500.0 ** (-i / a) for a in (16, 24) for i in range(a)]
    assert torch.equal(f, torch.tensor(want, dtype=torch.float64).float())
    f, scale = spark_rope_frequencies([n], base, "linear", 4.0)
    assert scale == 1.0
    assert torch.equal(f, torch.tensor([base ** (-i / n) / 4 for i in range(n)],
                                       dtype=torch.float64).float())
    f, _ = spark_rope_frequencies([n], base, "ntk", 4.0)
    assert f[0] == 1.0
    assert abs(f[-1].item() * 4 / base ** (-(n - 1) / n) - 1) < 1e-6
    assert spark_rope_frequencies([1], base, "ntk", 4.0)[0].tolist() == [1.0]


def test_yarn_frequencies():
    n, base, factor, original = 64, 10000.0, 8.0, 4096.0
    f, scale = spark_rope_frequencies([n], base, "yarn", factor, original)
    assert abs(scale - (0.1 * math.log(factor) + 1)) < 1e-15
    plain = [base ** (-i / n) for i in range(n)]
    seen = set()
    for i, p in enumerate(plain):
        turns = original * p / (2 * math.pi)
        got = f[i].item()
        if turns > 32 * base ** (1 / n):                  # a whole index above the ramp
            assert abs(got / p - 1) < 1e-6
            seen.add("kept")
        elif turns < base ** (-1 / n):
            assert abs(got / (p / factor) - 1) < 1e-6
            seen.add("stretched")
        else:
            assert p / factor * (1 - 1e-6) <= got <= p * (1 + 1e-6)
            seen.add("ramp")
    assert seen == {"kept", "stretched", "ramp"}
    f, scale = spark_rope_frequencies([n], base, "yarn", 1.0, original)
    assert scale == 1.0 and torch.allclose(f, torch.tensor(plain).float(), rtol=1e-6, atol=0)


def test_frequency_refusals():
    for args in (([4], 1.0), ([4], math.inf), ([-1], 10.0), ([], 10.0), ([4], 10.0, "linear", 0.5),
                 ([4], 10.0, "ntk", math.nan), ([4], 10.0, "yarn", 2.0, 0.0), ([1] * 5, 10.0)):
        with pytest.raises(SparkError):
            spark_rope_frequencies(*args)
    with pytest.raises(KeyError):
        spark_rope_frequencies([4], 10.0, "other")


def test_joint_sizes_and_refusals(L):
    a = (24, 60480, 128, 473, 473, 0.1)
    assert spark_bsa_workspace_size_joint(*a, 512) >= \
        spark_bsa_workspace_size_ctx(*a, 512) + spark_attend_dense_workspace_size(24, 512, 60480,
                                                                                  512, 128)
    assert spark_bsa_workspace_size_joint(*a, 0) == 0
    assert spark_bsa_workspace_size_joint(24, 60480, 96, 473, 473, 0.1, 512) == 0

    def joint(**kw):
        v = dict(Q=P, K=P, V=P, Qc=P, Kc=P, Vc=P, nc=77, dtype=0, H=2, N=1000, d=128, qp=P, kp=P,
                 qo=P, nqb=10, ko=P, nkb=10, ratio=0.2, out=P, out_c=P, ws=P, ws_bytes=1 << 20,
                 stream=None)
        v.update(kw)
        return L.spark_bsa_forward_joint(*v.values())

    assert joint(Qc=None) == INVALID
    assert joint(out_c=None) == INVALID
    assert joint(Kc=None) == INVALID
    assert joint(nc=0) == INVALID
    assert joint(out_c=ctypes.c_void_p(0x100004)) == INVALID
    assert joint(d=96) == UNSUPPORTED
    assert joint(ws_bytes=1024) == WORKSPACE
    assert joint(Q=None, ws_bytes=1 << 40) == INVALID
    assert joint(dtype=5, ws_bytes=1 << 40) == INVALID


def test_joint_outputs_over_inputs_are_refused(L):
    """By their bytes, not their first byte alone; what only touches is none of it.  A call that is
    not refused ends at the launch, as there is no GPU."""
    at = ctypes.c_void_p
    n, c = 2 * 1000 * 128 * 2, 2 * 77 * 128 * 2              # bytes of Q, K, V and of the context's

    def joint(**kw):
        v = dict(Q=at(0x1000000), K=at(0x2000000), V=at(0x3000000), Qc=at(0x4000000),
                 Kc=at(0x5000000), Vc=at(0x6000000), nc=77, dtype=0, H=2, N=1000, d=128, qp=P, kp=P,
                 qo=P, nqb=10, ko=P, nkb=10, ratio=0.2, out=at(0x7000000), out_c=at(0x8000000),
                 ws=at(0x9000000), ws_bytes=1 << 30, stream=None)
        v.update(kw)
        return L.spark_bsa_forward_joint(*v.values())

    if not torch.cuda.is_available():
        assert joint() not in (OK, INVALID)
        assert joint(out_c=at(0x4000000 - c), out=at(0x4000000 + c)) not in (OK, INVALID)
    for start in (0x4000000, 0x5000000, 0x6000000):
        for shift in (0, c - 16, 16 - c):
            assert joint(out_c=at(start + shift)) == INVALID
        for shift in (0, c - 16, 16 - n):
            assert joint(out=at(start + shift)) == INVALID
    for shift in (0, n - 16, 16 - c):
        assert joint(out_c=at(0x7000000 + shift)) == INVALID


def test_dense_outputs_over_inputs_are_refused(L):
    """As above."""
    at = ctypes.c_void_p
    nq, nk, nc = (2 * r * 128 * 2 for r in (300, 1000, 10))

    def attend(**kw):
        v = dict(Q=at(0x1000000), K=at(0x2000000), V=at(0x3000000), Kc=at(0x5000000),
                 Vc=at(0x6000000), lse=at(0x7000000), out=at(0x8000000), ws=at(0x9000000),
                 ws_bytes=1 << 30, ranges=at(0xa000000))
        return dense(L, **{**v, **kw})

    if not torch.cuda.is_available():
        assert attend() not in (OK, INVALID)
        assert attend(out=at(0x1000000 + nq), lse=at(0x2000000 + nk)) not in (OK, INVALID)
    for start, size in ((0x1000000, nq), (0x2000000, nk), (0x3000000, nk), (0x5000000, nc),
                        (0x6000000, nc), (0xa000000, 300 * 16)):
        for shift in (0, size - 16, 16 - nq):
            assert attend(out=at(start + shift)) == INVALID
        assert attend(lse=at(start + size - 4)) == INVALID
        assert attend(lse=at(start + 4 - 2 * 300 * 4)) == INVALID
    assert attend(lse=at(0x8000000 + nq - 4)) == INVALID
    assert attend(out_dtype=1, out=at(0x1000000 - 2 * nq + 16)) == INVALID


def test_binding_refuses_host_tensors_and_types():
    t = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        spark_attend_dense(t, t, t)
    with pytest.raises(ValueError, match="CUDA tensor"):
        spark_qk_norm_rope(t, t, t)
    with pytest.raises(TypeError, match="Q must be"):
        spark_qk_norm_rope([1, 2], t)
    with pytest.raises(TypeError, match="Q must be"):
        spark_attend_dense(None or [1], t, t)
    with pytest.raises(ValueError, match="CUDA tensor"):
        spark_attend_ranges(4, torch.zeros(2, dtype=torch.int32))
    perm = torch.zeros(1, 8, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        spark_bsa_forward_joint(t, t, t, t, t, t, perm, perm, perm[0], perm[0], 0.5)
