"""GPU tests of the dense attention over video and context keys and of the key ranges, against
the definition in 64 bits.

Tolerances, per output value, before any run: a probability is rounded to bf16 for the tensor
cores (at most half a step, 2^-8 of it) while the sum that divides it is not, so the weighted sum
is off by at most 2^-8 * A with A = sum_j p_j |v_j|; a bf16 output adds 2^-8 |out|.  The fp32 part:
a score is a sum of 128 products, each addition off by at most 2^-23 (truncated) of at most
sum |q k| sigma < 2^5 here, so 2^-11 at the very worst; it is held to 2^-12 of A, and the
log-sum-exp to 2^-12.
"""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _parity as P
from block_sparse_attention_gather_b200 import (
    DEVERR, spark_attend_dense, spark_attend_dense_workspace_size, spark_attend_ranges,
    spark_bsa_forward_ctx, spark_bsa_forward_joint, spark_bsa_get_wait_limit_ns,
    spark_bsa_read_error, spark_bsa_set_wait_limit_ns, spark_qk_norm_rope, spark_reblock,
    spark_rope_frequencies, workspace_views)
from test_gpu_parity import custom_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def inputs(seed, H, nq, nk, nc, d, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(n, s=1.0):
        return (torch.randn(H, n, d, generator=g, device=DEV) * s).to(BF)

    return dict(Q=rand(nq, scale), K=rand(nk), V=rand(nk), Kc=rand(nc) if nc else None,
                Vc=rand(nc) if nc else None)


def reference(x, ranges=None, heads=None):
    """(out, lse, sum p |v|) of the given heads in 64 bits."""
    H, nq, d = x["Q"].shape
    nk = x["K"].shape[1]
    outs = []
    for h in range(H) if heads is None else heads:
        k, v = x["K"][h].double(), x["V"][h].double()
        if x["Kc"] is not None:
            k, v = torch.cat([k, x["Kc"][h].double()]), torch.cat([v, x["Vc"][h].double()])
        s = x["Q"][h].double() @ k.T / math.sqrt(d)
        if ranges is not None:
            j = torch.arange(k.shape[0], device=DEV)
            r = ranges.long()[:, :, None]
            live = ((j >= r[:, 0]) & (j < r[:, 1]) & (j < nk)) | \
                ((j - nk >= r[:, 2].clamp(min=0)) & (j - nk < r[:, 3]))
            s = torch.where(live, s, torch.full_like(s, -math.inf))
        lse = torch.logsumexp(s, dim=1)
        p = torch.exp(s - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[:, None])
        # a masked value takes no part, whatever it holds
        v = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
        outs.append((p @ v, lse, p @ v.abs()))
    return [torch.stack(t) for t in zip(*outs)]


def check(x, out, lse, ranges=None, heads=None):
    ref, rl, A = reference(x, ranges, heads)
    if heads is not None:
        out, lse = out[list(heads)], lse[list(heads)]
    got = out.double()
    assert torch.isfinite(got).all()
    tol = (2.0 ** -8 + 2.0 ** -12) * A + (2.0 ** -8 * ref.abs() if out.dtype == BF else 0) + 1e-30
    worst = ((got - ref).abs() / tol).max().item()
    assert worst <= 1.0, f"output off by {worst:.2f} of its tolerance"
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert (got[empty] == 0).all()
    if (~empty).any():
        assert (lse.double() - rl)[~empty].abs().max().item() <= 2.0 ** -12


SIZES = [(1, 1, 1, 0, 128), (2, 1, 129, 0, 64), (3, 127, 300, 5, 128), (2, 128, 0, 77, 64),
         (1, 129, 1000, 1, 128), (2, 257, 511, 130, 64), (1, 300, 40000, 300, 128),
         (24, 1, 5000, 0, 128), (2, 513, 128, 128, 64), (2, 700, 2000, 0, 128),
         (5, 3, 20001, 77, 64)]


@pytest.mark.parametrize("H,nq,nk,nc,d", SIZES)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_all_keys(H, nq, nk, nc, d, dtype):
    x = inputs(11 + nq, H, nq, nk, nc, d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = spark_attend_dense(**x, out_dtype=dtype, err=err)
    assert spark_bsa_read_error(err) == 0
    check(x, out, lse)


def random_ranges(seed, nq, nk, nc):
    """Ranges of every kind: whole, short, one key, empty, reversed, past both ends."""
    rng = np.random.default_rng(seed)
    r = np.zeros((nq, 4), dtype=np.int64)
    for i in range(nq):
        for at, n in ((0, nk), (2, nc)):
            a, b = sorted(rng.integers(0, n + 1, 2))
            kind = rng.integers(0, 6)
            if kind == 0:
                a, b = 0, n
            elif kind == 1:
                b = min(a + 1, n)
            elif kind == 2:
                b = a
            elif kind == 3:
                a, b = b, a
            elif kind == 4:
                a, b = -5, n + 1000
            r[i, at], r[i, at + 1] = a, b
    return torch.from_numpy(r.astype(np.int32)).to(DEV)


@pytest.mark.parametrize("H,nq,nk,nc,d", SIZES)
def test_any_ranges(H, nq, nk, nc, d):
    x = inputs(23 + nq, H, nq, nk, nc, d)
    r = random_ranges(nq, nq, nk, nc)
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    check(x, out, lse, r)


@pytest.mark.parametrize("nq", [1, 100, 300])
def test_every_row_empty(nq):
    x = inputs(5, 2, nq, 700, 30, 128)
    r = torch.tensor([[9, 9, 30, 30]], dtype=torch.int32, device=DEV).repeat(nq, 1)
    out, lse = spark_attend_dense(**x, ranges=r)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("nq", [1, 200])
def test_no_keys_at_all(nq):
    x = inputs(6, 2, nq, 0, 0, 64)
    out, lse = spark_attend_dense(**x)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("nq", [3, 128, 300])
@pytest.mark.parametrize("step", [0.05, 3.0])
def test_maximum_that_keeps_growing(nq, step):
    """Scores that rise along the keys: the running reference has to follow."""
    H, nk, d = 2, 1500, 128
    x = inputs(7, H, nq, nk, 40, d)
    u = torch.ones(d, device=DEV) / math.sqrt(d)
    x["Q"] = (x["Q"].float() * 0.1 + 4 * u).to(BF)
    ramp = torch.linspace(0, step * 12, nk, device=DEV)[None, :, None]
    x["K"] = (x["K"].float() * 0.1 + ramp * u * math.sqrt(d)).to(BF)
    out, lse = spark_attend_dense(**x, out_dtype=torch.float32)
    ref, rl, A = reference(x)
    # scores reach 144: their fp32 sums are off by up to 2^-23 * 128 * 144 < 2^-8 at the worst
    assert ((out.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -7) * A).all()
    assert (lse.double() - rl).abs().max() <= 2.0 ** -8


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq", [1, 130, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masked_places_may_hold_anything(nq, d, bad):
    x = inputs(8, 2, nq, 700, 200, d)
    lo, hi, clo, chi = 130, 601, 3, 77
    for k in ("K", "V"):
        x[k][:, :lo] = bad
        x[k][:, hi:] = bad
        x[k + "c"][:, :clo] = bad
        x[k + "c"][:, chi:] = bad
    r = torch.tensor([[lo, hi, clo, chi]], dtype=torch.int32, device=DEV).repeat(nq, 1)
    if nq > 2:
        r[1] = torch.tensor([5, 5, 9, 2])                  # a row of nothing
        r[2] = torch.tensor([lo + 7, lo + 8, 0, 0])        # a row of one key
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    for k in ("K", "V"):
        x[k][:, :lo] = 0
        x[k][:, hi:] = 0
        x[k + "c"][:, :clo] = 0
        x[k + "c"][:, chi:] = 0
    check(x, out, lse, r)


@pytest.mark.parametrize("d", [64, 128])
def test_masked_values_as_large_as_the_type_holds(d):
    """Keys that some rows of a tile see and others mask, with values up to bf16's largest: nothing of
    them may reach the rows that mask them."""
    x = inputs(17, 2, 300, 700, 130, d)
    r = torch.zeros(300, 4, dtype=torch.int32, device=DEV)
    r[:, 1], r[:, 3] = 500, 60
    r[::2] = torch.tensor([200, 700, 60, 130], device=DEV, dtype=torch.int32)
    large = torch.finfo(BF).max
    x["V"][:, 500:], x["Vc"][:, 60:] = large / 2 ** 20, -large / 2 ** 20
    x["V"][:, :200], x["Vc"][:, :60] = large, -large       # the even rows' masked keys
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    for t, n in (("V", 200), ("Vc", 60)):
        x[t][:, :n] = 0
    even = dict(x, Q=x["Q"][:, ::2].contiguous())
    check(even, out[:, ::2], lse[:, ::2], r[::2].contiguous())
    x["V"][:, 500:], x["Vc"][:, 60:] = large, -large       # and the odd rows'
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    x["V"][:, 500:], x["Vc"][:, 60:] = 0, 0
    odd = dict(x, Q=x["Q"][:, 1::2].contiguous())
    check(odd, out[:, 1::2], lse[:, 1::2], r[1::2].contiguous())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("order", ["up", "down", "mixed", "holes"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_padding_between_the_segments_may_hold_anything(d, order, bad):
    """Keys in segments with padding between them, several segments to a tile of queries, rows of
    nothing among them."""
    nq, nk, nc = 300, 2000, 260
    x = inputs(18, 2, nq, nk, nc, d)
    starts = list(range(10, 1900, 190))                    # 10 segments, 30 rows each
    lens = [150, 190, 1, 127, 128, 129, 64, 100, 33, 180]
    which = list(range(10))
    if order == "down":
        which = which[::-1]
    if order == "mixed":
        which = [3, 0, 7, 7, 1, 9, 2, 8, 4, 6]
    r = torch.zeros(nq, 4, dtype=torch.int32)
    for i, b in enumerate(which):
        r[30 * i:30 * i + 30] = torch.tensor([starts[b], starts[b] + lens[b], 26 * b, 26 * b + 20])
    if order == "holes":
        r[::3, :2] = 0
        r[1::3, 2:] = 7
        r[125:131] = 0
    used = torch.zeros(nk, dtype=torch.bool), torch.zeros(nc, dtype=torch.bool)
    for a, b, c, e in r.tolist():
        used[0][a:b], used[1][c:e] = True, True
    for t, u in (("K", 0), ("V", 0), ("Kc", 1), ("Vc", 1)):
        x[t][:, (~used[u]).to(DEV)] = bad
    r = r.to(DEV)
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    for t, u in (("K", 0), ("V", 0), ("Kc", 1), ("Vc", 1)):
        x[t][:, (~used[u]).to(DEV)] = 0
    check(x, out, lse, r)


def test_range_bounds_of_any_int32():
    low, high = -2 ** 31, 2 ** 31 - 1
    x = inputs(19, 2, 5, 900, 300, 128)
    r = torch.tensor([[low, 20, low, high], [800, high, low, low], [high, low, 100, high],
                      [low, high, high, high], [high, high, low, 1]], dtype=torch.int32, device=DEV)
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    check(x, out, lse, r.clamp(min=0))
    r = r[:3].contiguous()
    r[0, 1] = r[1, 3] = r[2, 1] = 20                       # a gap between keys 20 and 800
    x["Q"] = x["Q"][:, :3].contiguous()
    x["V"][:, 20:800] = math.nan
    r[2, 0] = low
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    x["V"][:, 20:800] = 0
    check(x, out, lse, r.clamp(min=0))


def test_nan_in_a_live_key_reaches_its_rows_only():
    x = inputs(9, 1, 2, 600, 0, 128)
    x["K"][0, 500] = math.nan
    r = torch.tensor([[0, 600, 0, 0], [0, 400, 0, 0]], dtype=torch.int32, device=DEV)
    out, lse = spark_attend_dense(**x, ranges=r)
    assert torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0])
    x["K"][0, 500] = 0
    ref, rl, A = reference(x, r)
    assert ((out[0, 1].double() - ref[0, 1]).abs() <= 2.0 ** -7 * A[0, 1] + 1e-6).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nk", [256, 4000])
@pytest.mark.parametrize("where", ["K", "Q", "inf"])
def test_nan_row_stays_one_past_its_last_key(nk, d, where):
    """Row 0's keys end a tile (and more) before those of the row beside it, in one slice of the keys
    and in several: the tiles where it sees nothing must not make it a row without keys."""
    x = inputs(70, 1, 2, nk, 0, d)
    if where == "Q":
        x["Q"][0, 0, 7] = math.nan
    elif where == "K":
        x["K"][0, 5] = math.nan
    else:
        x["K"][0, 5], x["Q"][0, 0] = math.inf, x["Q"][0, 0].abs() + 0.5
    r = torch.tensor([[0, 100, 0, 0], [64, nk, 0, 0]], dtype=torch.int32, device=DEV)
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    assert torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0])
    x["K"][0, 5] = 0
    other = dict(x, Q=x["Q"][:, 1:].contiguous())
    check(other, out[:, 1:], lse[:, 1:], r[1:].contiguous())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nk", [700, 9000])
@pytest.mark.parametrize("step", [8.0, 14.0, 16.0, 60.0])
def test_large_values_under_scores_that_rise(nk, d, step):
    """Values of 2^118 and scores `step` nats higher (14: 20 powers of two) from key 300 on, and again
    from key 500 on.  The definition is finite, and so is an fp32 sum of p |v| with p <= 1:
    |v| < 2^118 * 8, and no 2^14 keys make it 2^128 unless they all have p near 1.  A score is one
    product, exact but for its scale: 2^-22 of 121 is under 2^-15."""
    g = torch.Generator(device=DEV).manual_seed(71)
    level = torch.zeros(nk, device=DEV)
    level[300:] += step
    level[500:] += step
    level = level + 0.3 * torch.randn(2, nk, generator=g, device=DEV)
    Q, K = torch.zeros(2, 40, d, device=DEV), torch.zeros(2, nk, d, device=DEV)
    Q[..., 0] = 16
    K[..., 0] = level * math.sqrt(d) / 16
    V = torch.randn(2, nk, d, generator=g, device=DEV).clamp(-8, 8) * 2.0 ** 118
    x = dict(Q=Q.to(BF), K=K.to(BF), V=V.to(BF), Kc=None, Vc=None)
    out, lse = spark_attend_dense(**x, out_dtype=torch.float32)
    check(x, out, lse)


@pytest.mark.parametrize("nats", [20, 60, 88, 100, 150, 200])
@pytest.mark.parametrize("tile", [0, 1, 4])
@pytest.mark.parametrize("far", [1, -1])
def test_one_key_far_above_the_others(nats, tile, far):
    """Row i's own key, at column i of the tile, exceeds all it saw before by up to 289 powers of
    two (or is that far below): every column of a tile, whatever computes its exponential."""
    H, n, d = 1, 900, 128
    g = torch.Generator(device=DEV).manual_seed(nats)
    eye = torch.eye(128, device=DEV)
    Q = (16 * eye)[None].to(BF)
    K = torch.zeros(H, n, d, device=DEV)
    K[:, 128 * tile:128 * tile + 128] = far * nats * math.sqrt(128) / 16 * eye
    x = dict(Q=Q, K=K.to(BF), V=torch.randn(H, n, d, generator=g, device=DEV).to(BF), Kc=None,
             Vc=None)
    out, lse = spark_attend_dense(**x, out_dtype=torch.float32)
    # one product per score, exact in fp32 but for its scale: 2^-22 of 200 is under 2^-14
    check(x, out, lse)


@pytest.mark.parametrize("nats", [20, 88, 100, 150])
@pytest.mark.parametrize("tile", [0, 1, 3])
def test_one_row_alone_meets_a_far_key(nats, tile):
    """As above with nothing else in the row's warp that would have the tile looked at again."""
    d, n = 128, 600
    g = torch.Generator(device=DEV).manual_seed(nats)
    V = torch.randn(1, n, d, generator=g, device=DEV).to(BF)
    Q = torch.zeros(1, 1, d, device=DEV)
    Q[..., 0] = 16
    Q = Q.to(BF)
    for j in range(128):
        K = torch.zeros(1, n, d, device=DEV)
        K[0, 128 * tile + j, 0] = nats * math.sqrt(128) / 16
        K = K.to(BF)
        out, lse = spark_attend_dense(Q, K, V, out_dtype=torch.float32)
        check(dict(Q=Q, K=K, V=V, Kc=None, Vc=None), out, lse)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("tile", [0, 1, 3])
def test_bad_score_at_every_column(bad, tile):
    x = inputs(16, 1, 3, 700, 0, 128)
    x["Q"] = x["Q"].abs() + 0.5
    keep = x["K"].clone()
    for j in range(128):
        x["K"] = keep.clone()
        x["K"][0, 128 * tile + j] = bad
        out, lse = spark_attend_dense(**x)
        assert torch.isnan(out).all() and torch.isnan(lse).all(), j


def test_keys_past_32_bit_offsets():
    """4.6 GB of keys: byte and element offsets beyond 2^32 and 2^31."""
    H, nk, d = 3, 6_000_000, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    K = torch.zeros(H, nk, d, dtype=BF, device=DEV)
    V = torch.zeros(H, nk, d, dtype=BF, device=DEV)
    n = 1000
    K[:, -n:] = torch.randn(H, n, d, generator=g, device=DEV).to(BF)
    V[:, -n:] = torch.randn(H, n, d, generator=g, device=DEV).to(BF)
    Q = torch.randn(H, 2, d, generator=g, device=DEV).to(BF)
    r = torch.tensor([[nk - n, nk, 0, 0], [nk - 1, nk, 0, 0]], dtype=torch.int32, device=DEV)
    out, lse = spark_attend_dense(Q, K, V, ranges=r, out_dtype=torch.float32)
    x = dict(Q=Q, K=K[:, -n:].contiguous(), V=V[:, -n:].contiguous(), Kc=None, Vc=None)
    r2 = torch.tensor([[0, n, 0, 0], [n - 1, n, 0, 0]], dtype=torch.int32, device=DEV)
    check(x, out, lse, r2)


def test_results_are_deterministic_and_workspace_independent():
    x = inputs(10, 4, 77, 9000, 77, 128)
    size = spark_attend_dense_workspace_size(4, 77, 9000, 77, 128)
    a = spark_attend_dense(**x)
    ws = torch.full((size + 1024,), 255, dtype=torch.uint8, device=DEV)
    b = spark_attend_dense(**x, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("nq", [1, 300])
def test_on_another_stream_and_in_graphs_that_share_a_workspace(nq):
    x = inputs(12, 2, nq, 9000, 33, 128)
    y = inputs(13, 2, nq, 9000, 33, 128)
    want = [spark_attend_dense(**t) for t in (x, y)]
    size = spark_attend_dense_workspace_size(2, nq, 9000, 33, 128)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    outs = [(torch.empty_like(w[0]), torch.empty_like(w[1])) for w in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    spark_attend_dense(**x, out=outs[0][0], lse=outs[0][1], workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(outs[0][0], want[0][0])
    graphs = []
    for t, (o, l) in zip((x, y), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            spark_attend_dense(**t, out=o, lse=l, workspace=ws)
        graphs.append(graph)
    for o, l in outs:
        o.zero_(), l.zero_()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (o, l), w in zip(outs, want):
        assert torch.equal(o, w[0]) and torch.equal(l, w[1])


FIRST_CALL = """
import torch
from block_sparse_attention_gather_b200 import spark_attend_dense
Q, K, V = (torch.randn(2, n, 128, device="cuda").bfloat16() for n in (3, 9000, 9000))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out, lse = spark_attend_dense(Q, K, V)
graph.replay()
want, _ = spark_attend_dense(Q, K, V)
torch.cuda.synchronize()
assert torch.equal(out, want)
"""


def test_first_call_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True,
                         text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-2000:]


def test_two_streams_at_once():
    """Calls that overlap on the GPU, each with a workspace of its own."""
    xs = [inputs(40 + i, 2, 9 + 200 * i, 20000, 50, 128) for i in range(2)]
    want = [spark_attend_dense(**x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got[i].append(spark_attend_dense(**x))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(o, w[0]) and torch.equal(l, w[1]) for o, l in g)


def test_calls_on_given_streams_without_workspaces():
    """stream= alone: the calls' own workspaces and outputs are nobody else's while they run, however
    long they wait for their streams."""
    xs = [inputs(50 + i, 2, 9, 9000, 33, 128) for i in range(2)]
    want = [spark_attend_dense(**x) for x in xs]
    size = spark_attend_dense_workspace_size(2, 9, 9000, 33, 128)
    assert size > 256                                      # split: partial sums go through it
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        torch.cuda.synchronize()
        for s in streams:
            with torch.cuda.stream(s):
                torch.cuda._sleep(10_000_000)              # a few milliseconds
        got = [spark_attend_dense(**x, stream=s) for x, s in zip(xs, streams)]
        other = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
                 for n in 2 * [size, want[0][0].nbytes, want[0][1].nbytes]]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
        assert all((t == 255).all() for t in other)


def test_captured_calls_on_given_streams_without_workspaces():
    xs = [inputs(52 + i, 2, 9, 9000, 33, 128) for i in range(2)]
    want = [spark_attend_dense(**x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for s in streams:
            s.wait_stream(main)
        got = [spark_attend_dense(**x, stream=s) for x, s in zip(xs, streams)]
        for s in streams:
            main.wait_stream(s)
        copies = [[t.clone() for t in g] for g in got]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(copies, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("H,nq,nk", [(2, 7, 9000), (8, 300, 300), (1, 128, 128)])
def test_calls_that_feed_each_other(H, nq, nk):
    """Each call's output is the next one's queries, in the same buffers: kernels may be set up
    before the one ahead of them ends, but must not read or write ahead of it."""
    x = inputs(60, H, nq, nk, 33, 128)
    size = spark_attend_dense_workspace_size(H, nq, nk, 33, 128)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    q, outs = x.pop("Q"), []
    for sync in (True, False):
        bufs = [q.clone(), torch.empty_like(q)]
        for i in range(30):
            spark_attend_dense(bufs[i % 2], **x, out=bufs[(i + 1) % 2], workspace=ws)
            if sync:
                torch.cuda.synchronize()
        outs.append(bufs[0].clone())
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("nq", [5, 300])
def test_expired_wait_is_flagged_and_leaves_the_context_usable(nq):
    x = inputs(14, 2, nq, 3000, 10, 128)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    old = spark_bsa_get_wait_limit_ns()
    try:
        spark_bsa_set_wait_limit_ns(0)
        spark_attend_dense(**x, err=err)
        torch.cuda.synchronize()
    finally:
        spark_bsa_set_wait_limit_ns(old)
    assert err.item() == DEVERR["timeout"]
    err.zero_()
    out, lse = spark_attend_dense(**x, err=err)
    assert spark_bsa_read_error(err) == 0
    check(x, out, lse)


# ------------------------------------------------------------------------------ key ranges

def ranges_reference(nq, q, k, c, prefix, causal):
    out = np.zeros((nq, 4), dtype=np.int32)
    for b in range(len(q) - 1):
        for i in range(q[b], min(q[b + 1], nq)):
            if k is not None:
                out[i, :2] = k[b], k[b + 1]
            if c is not None:
                lc, end = c[b + 1] - c[b], c[b + 1] - c[b]
                if causal:
                    seen = i - q[b] + 1 + lc - (q[b + 1] - q[b])
                    end = min(max(seen, prefix[b] if prefix is not None else 0, 0), lc)
                out[i, 2:] = c[b], c[b] + end
    return out


@pytest.mark.parametrize("nseg,rows,pad", [(1, 1, 0), (1, 50, 3), (7, 300, 0), (64, 40, 9),
                                           (1000, 5000, 100)])
@pytest.mark.parametrize("causal", [False, True])
def test_ranges_of_segments(nseg, rows, pad, causal):
    rng = np.random.default_rng(nseg + rows)

    def offsets(total):
        return np.concatenate([[0], np.sort(rng.integers(0, total + 1, nseg - 1)), [total]])

    q, k, c = offsets(rows), offsets(70000), offsets(rows + 20)
    prefix = rng.integers(-3, 40, nseg)
    dev = [torch.tensor(t, dtype=torch.int32, device=DEV) for t in (q, k, c, prefix)]
    for use in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 0)):
        kk, cc = (dev[1] if use[0] else None), (dev[2] if use[1] else None)
        pp = dev[3] if use[2] and causal else None
        got = spark_attend_ranges(rows + pad, dev[0], kk, cc, prefix=pp, causal=causal)
        want = ranges_reference(rows + pad, q, k if use[0] else None, c if use[1] else None,
                                prefix if pp is not None else None, causal)
        assert np.array_equal(got.cpu().numpy(), want)


def test_ranges_of_the_most_segments():
    """2^30 segments, empty but for the first and the last: the search's bounds add up to 2^31."""
    n = 1 << 30
    q = torch.full((n + 1,), 2, dtype=torch.int32, device=DEV)          # 4.3 GB
    q[0], q[-1] = 0, 5
    got = spark_attend_ranges(7, q, None, q)
    assert got.tolist() == [[0, 0, 0, 2]] * 2 + [[0, 0, 2, 5]] * 3 + [[0, 0, 0, 0]] * 2


def test_ranges_refuse_decreasing_key_offsets_in_the_error_word():
    q = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    k = torch.tensor([0, 9, 5], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = spark_attend_ranges(4, q, k, err=err)
    assert err.item() == DEVERR["offsets"]
    assert got.tolist() == [[0, 9, 0, 0]] * 2 + [[0, 0, 0, 0]] * 2


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_packed_prompts_equal_one_call_per_clip(d, causal):
    """Segments of every length, zero and one among them, and rows of padding at the end."""
    ql, kl = [77, 0, 1, 200, 130], [500, 64, 1, 0, 1303]
    q = torch.tensor(np.cumsum([0] + ql), dtype=torch.int32, device=DEV)
    k = torch.tensor(np.cumsum([0] + kl), dtype=torch.int32, device=DEV)
    nq = sum(ql) + 7
    x = inputs(15, 2, nq, sum(kl), nq, d)
    for t in ("Kc", "Vc"):
        x[t][:, sum(ql):] = math.nan                       # padding of the prompts
    r = spark_attend_ranges(nq, q, k, q, causal=causal)
    out, lse = spark_attend_dense(**x, ranges=r, out_dtype=torch.float32)
    for t in ("Kc", "Vc"):
        x[t][:, sum(ql):] = 0
    check(x, out, lse, r)
    assert (out[:, sum(ql):] == 0).all()


# ------------------------------------------------------------- together, as they are used

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nc", [1, 77, 300])
def test_joint_forward(dtype, nc):
    x = custom_inputs(31, 2, 1500, 128, dtype, 30, 128)
    H, N, d = x["Q"].shape
    g = torch.Generator().manual_seed(4)
    for n in ("Qc", "Kc", "Vc"):
        x[n] = torch.randn(H, nc, d, generator=g).to(x["Q"].dtype).to(DEV)
    perms = (x["q_perm"], x["k_perm"], x["q_offsets"], x["k_offsets"])
    out, out_c, ws, layout = spark_bsa_forward_joint(x["Q"], x["K"], x["V"], x["Qc"], x["Kc"],
                                                     x["Vc"], *perms, 0.2)
    views = workspace_views(ws, layout, H, N, d, x["q_offsets"].numel() - 1,
                            x["k_offsets"].numel() - 1)
    assert spark_bsa_read_error(views["err"]) == 0
    want, _, _ = spark_bsa_forward_ctx(x["Q"], x["K"], x["V"], x["Kc"], x["Vc"], *perms, 0.2)
    assert torch.equal(out, want)
    # the context queries against the definition, on the bf16 values the kernels see
    b = {n: x[n].to(BF) for n in ("K", "V", "Kc", "Vc")}
    b["Q"] = x["Qc"].to(BF)
    ref, _, A = reference(b)
    tol = (2.0 ** -8 + 2.0 ** -12) * A + (2.0 ** -8 * ref.abs() if dtype == "bf16" else 0)
    assert out_c.dtype == x["Q"].dtype
    assert ((out_c.double() - ref).abs() <= tol).all()


def test_projection_to_joint_attention():
    """A fused projection's output through norm and rotation, the partitioner and the joint
    attention, against the same steps in 64 bits where they are not the sparse call itself."""
    H, N, nc, d = 2, 1280, 77, 128
    g = torch.Generator(device=DEV).manual_seed(21)
    video = torch.randn(N, 3, H, d, generator=g, device=DEV).to(BF)
    text = torch.randn(nc, 3, H, d, generator=g, device=DEV).to(BF)
    w = [(1 + 0.1 * torch.randn(d, generator=g, device=DEV)) for _ in range(2)]
    axes = [16, 24, 24]
    freq, scale = spark_rope_frequencies(axes)
    pos = torch.stack(torch.meshgrid(*(torch.arange(n) for n in (5, 16, 16)), indexing="ij"),
                      dim=-1).reshape(-1, 3).int().to(DEV)
    Q, K, V = (video[:, i].transpose(0, 1) for i in range(3))
    Q, K, V = spark_qk_norm_rope(Q, K, V, *w, positions=pos, inv_freq=freq.to(DEV),
                                 axis_pairs=axes, interleaved=True, rope_scale=scale)
    Qc, Kc, Vc = (text[:, i].transpose(0, 1) for i in range(3))
    Qc, Kc, Vc = spark_qk_norm_rope(Qc, Kc, Vc, *w)
    q_perm, k_perm, offsets = spark_reblock(Q, K, block=128)
    out, out_c, ws, layout = spark_bsa_forward_joint(Q, K, V, Qc, Kc, Vc, q_perm, k_perm, offsets,
                                                     offsets, 1.0)
    views = workspace_views(ws, layout, H, N, d, offsets.numel() - 1, offsets.numel() - 1)
    assert spark_bsa_read_error(views["err"]) == 0
    # ratio 1: every block is exact, so the video rows are dense attention too
    dense, lse = spark_attend_dense(Q, K, V, Kc, Vc, out_dtype=torch.float32)
    check(dict(Q=Q, K=K, V=V, Kc=Kc, Vc=Vc), dense, lse)
    P.compare_out(P.to64(out), P.to64(dense), "video rows at ratio 1")
    ref, _, A = reference(dict(Q=Qc, K=K, V=V, Kc=Kc, Vc=Vc))
    assert ((out_c.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -12) * A + 2.0 ** -8 * ref.abs()).all()


def test_binding_refusals():
    x = inputs(50, 2, 5, 40, 7, 64)
    r = torch.zeros(5, 4, dtype=torch.int32, device=DEV)
    good = dict(x, ranges=r)
    spark_attend_dense(**good)
    for name, bad, kind in (
            ("Q", x["Q"].float(), TypeError), ("Q", x["Q"][:, ::2], ValueError),
            ("Q", x["Q"][0], ValueError), ("K", x["K"].cpu(), ValueError),
            ("K", x["K"][:1], ValueError), ("V", x["V"][:, :9].contiguous(), ValueError),
            ("V", None, TypeError), ("Kc", x["Kc"].half(), TypeError), ("Vc", None, TypeError),
            ("Vc", x["Vc"][:, :3].contiguous(), ValueError), ("ranges", r.long(), TypeError),
            ("ranges", r[:4], ValueError), ("out", x["Q"].half(), TypeError),
            ("out", x["Q"][:1].contiguous(), ValueError), ("lse", r, TypeError),
            ("lse", torch.zeros(2, 4, device=DEV), ValueError), ("workspace", r, TypeError),
            ("err", torch.zeros(1, device=DEV), TypeError)):
        with pytest.raises((kind,) if kind is not TypeError else (TypeError, ValueError)):
            spark_attend_dense(**{**good, name: bad})
    q = torch.tensor([0, 3, 5], dtype=torch.int32, device=DEV)
    for args, kw in (((5, q.long()), {}), ((5, q, q[:2]), {}), ((5, q, q.cpu()), {}),
                     ((5, q, None, q), dict(prefix=q, causal=True)),
                     ((5, q, None, q), dict(prefix=q[:2])), ((5, q), dict(ranges=r[:4])),
                     ((5, q, [1, 2, 3]), {})):
        with pytest.raises((TypeError, ValueError)):
            spark_attend_ranges(*args, **kw)


def test_captured_among_copies_and_on_two_streams():
    """A graph whose calls follow a memset and a copy, and join branches of two streams."""
    x = inputs(20, 4, 130, 1500, 0, 128)
    w = torch.rand(128, device=DEV) + 0.5
    pos = torch.arange(1500, device=DEV, dtype=torch.int32)[:, None]
    freq = spark_rope_frequencies([64])[0].to(DEV)
    q, k, k2, v = x["Q"].clone(), torch.empty_like(x["K"]), torch.empty_like(x["K"]), x["V"].clone()
    r = torch.empty(130, 4, dtype=torch.int32, device=DEV)
    qo = torch.tensor([0, 50, 130], dtype=torch.int32, device=DEV)
    ko = torch.tensor([0, 700, 1500], dtype=torch.int32, device=DEV)
    out = [torch.empty_like(q) for _ in range(3)]
    side = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        k.zero_()
        spark_qk_norm_rope(x["K"], None, None, w, None, 1e-6, pos, freq, [64], Q_out=k)
        spark_attend_dense(q, k, v, out=out[0])
        side.wait_stream(main)
        with torch.cuda.stream(side):
            spark_qk_norm_rope(k, None, None, w, None, 1e-6, pos, freq, [64], Q_out=k2)
            spark_attend_ranges(130, qo, ko, ranges=r)
            spark_attend_dense(out[0], k2, v, out=out[1])
        spark_attend_dense(out[0], k, v, out=out[2])
        main.wait_stream(side)
        spark_attend_dense(out[1], k2, out[2].repeat(1, 12, 1)[:, :1500].contiguous(), ranges=r,
                           out=q)
        k2.copy_(k)
        spark_attend_dense(q, k2, v, out=out[0])

    start = x["Q"].clone()
    want = []
    for _ in range(3):
        work()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (q, *out)])
    q.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((q, *out), want[i]):
            assert torch.isfinite(a).all() and torch.equal(a, b), i
