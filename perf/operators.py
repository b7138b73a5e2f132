"""What is measured of the operators next to the block-sparse forward, and their plain forms.

Three operators that a caller of the block-sparse attention needs around it:

* ``norm_rope`` - Q and K as a projection leaves them (token-major, strided views) normalised per
  head, rotated by their positions and laid out ``[H, N, d]`` in one pass, V laid out with them.
* ``ranges``    - the key ranges of every query, from segment offsets on the device: documents,
  prefixes and causal prompts.
* ``dense``     - dense attention of some queries (the context tokens, or every token of a dense
  layer) over the video keys and the context keys, under such ranges, with the rows' log-sum-exp.

With ``own`` false ``run`` computes an operator with elementary torch operations in 32 bits
(angles in 64); with ``own`` true it calls the library.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one new token of a text stream at a far position, its fused projection's row
        dict(name="rope-one-token", op="norm_rope", N=1, H=16, d=128, dtype="bf16", layout="half",
             axes="64", far=1000000, packed=True, with_v=True, norm=True, scale=1.0),
        # a 77-token prompt in fp32, a part of each head rotated, scaled for a long context
        dict(name="rope-prompt-fp32", op="norm_rope", N=77, H=8, d=64, dtype="fp32",
             layout="half", axes="16", far=40000, packed=False, with_v=False, norm=True,
             scale=1.1386),
        # a 16384-token clip: time, height and width axes, interleaved pairs
        dict(name="rope-clip", op="norm_rope", N=16384, H=8, d=128, dtype="bf16",
             layout="interleaved", axes="16,24,24", far=84, packed=True, with_v=True, norm=True,
             scale=1.0),
        # every token of a 384p video
        dict(name="rope-384p", op="norm_rope", N=60480, H=20, d=128, dtype="bf16",
             layout="interleaved", axes="16,24,24", far=60, packed=True, with_v=True, norm=True,
             scale=1.0),
        # key ranges of four clips' prompts, padded
        dict(name="ranges-prompts", op="ranges", q="77,64,120,33", k="6048,4033,5000,1303",
             c="77,64,120,33", prefix="", causal=False, pad=6),
        # key ranges of every token of many packed documents, prefix and causal
        dict(name="ranges-documents", op="ranges", q="241*1000,920", k="", c="241*1000,920",
             prefix="16", causal=True, pad=0),
        # one summary token over a 384p video
        dict(name="dense-one-query", op="dense", H=24, d=128, q="1", k="60480", c="",
             mask="none", pad=0),
        # a prompt's queries over the smallest workload with its context
        dict(name="dense-tiny", op="dense", H=8, d=64, q="77", k="1024", c="77", mask="none",
             pad=0),
        # four clips and their prompts packed into one call, rows of padding at the end
        dict(name="dense-packed-prompts", op="dense", H=8, d=128, q="77,64,120,33",
             k="6048,4033,5000,1303", c="77,64,120,33", mask="segments", pad=6),
        # a long prompt: a bidirectional prefix, causal after it, no video keys
        dict(name="dense-prefix", op="dense", H=16, d=128, q="8191", k="", c="8191",
             mask="causal", prefix="1000", pad=0),
        # the context queries of the 768p workload: 512 rows over every video and context key
        dict(name="dense-context-768p", op="dense", H=24, d=128, q="512", k="241920", c="512",
             mask="none", pad=0),
        # a dense layer over half the frames of a 384p video
        dict(name="dense-layer", op="dense", H=24, d=128, q="30240", k="30240", c="", mask="none",
             pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _pieces(rng, total, n):
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _text(lens):
    return ",".join(str(v) for v in lens)


def draw(rng):
    op = rng.choice(["norm_rope", "dense", "dense", "ranges"])
    if op == "norm_rope":
        d = rng.choice([64, 128])
        H = rng.randint(1, 24)
        N = min(_log(rng, 1, 60480), 60480 * 20 * 128 // (H * d))
        pairs = rng.choice([d // 2, d // 2, d // 4, rng.randint(1, d // 2)])
        axes = [p for p in _pieces(rng, pairs, rng.randint(1, 3)) if p > 0]
        return dict(op=op, N=N, H=H, d=d, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    layout=rng.choice(["half", "interleaved"]), axes=_text(axes),
                    far=_log(rng, 30, 1000000), packed=rng.random() < 0.7,
                    with_v=rng.random() < 0.6, norm=rng.random() < 0.8,
                    scale=rng.choice([1.0, 1.2079]))
    if op == "ranges":
        n = _log(rng, 1, 1000)
        q = _pieces(rng, _log(rng, n, 241920), n)
        causal = rng.random() < 0.5
        k = _pieces(rng, rng.randint(1, 241920), n) if rng.random() < 0.6 else []
        return dict(op=op, q=_text(q), k=_text(k), c=_text(q), causal=causal,
                    prefix=str(rng.randint(0, 64)) if causal else "", pad=rng.randint(0, 40))
    H, d = rng.randint(1, 24), rng.choice([64, 128, 128])
    mask = rng.choice(["none", "segments", "causal"])
    nk = _log(rng, 1, 120000)
    if mask == "none":
        nq = _log(rng, 1, 8000)
        return dict(op=op, H=H, d=d, q=str(nq), k=str(nk), c=str(rng.choice([0, 1, 77, 300, 512])),
                    mask=mask, pad=0)
    n = rng.randint(1, 6)
    nq = _log(rng, n, 6000)
    q = _pieces(rng, nq, n)
    k = _pieces(rng, nk, n) if rng.random() < 0.7 else []
    case = dict(op=op, H=H, d=d, q=_text(q), k=_text(k), c=_text(q), mask=mask,
                pad=rng.randint(0, 9))
    if mask == "causal":
        case["prefix"] = str(rng.randint(0, max(1, nq // n)))
    return case


# ------------------------------------------------------------------------------------ inputs

def _lens(text):
    out = []
    for part in text.split(","):
        if part:
            v, _, times = part.partition("*")
            out += [int(v)] * (int(times) if times else 1)
    return out


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(np.asarray(lens, dtype=np.int64))])


def _rope_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    H, N, d, dt = case["H"], case["N"], case["d"], DTYPES[case["dtype"]]
    if case["packed"]:
        # a fused projection's output, token-major: views of one tensor, no copy
        x = torch.randn(N, 3, H, d, generator=g, device=DEV)
        x = (x * (0.5 + torch.rand(3, H, 1, generator=g, device=DEV))).to(dt)
        Q, K, V = (x[:, i].transpose(0, 1) for i in range(3))
    else:
        Q, K, V = ((torch.randn(H, N, d, generator=g, device=DEV) * 1.3).to(dt) for _ in range(3))
    axes = [int(a) for a in case["axes"].split(",")]
    wq = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
    wk = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
    pos = torch.randint(0, case["far"], (N, len(axes)), generator=g, device=DEV, dtype=torch.int32)
    freq = torch.cat([10000.0 ** (-torch.arange(a, dtype=torch.float64) / a) for a in axes])
    return dict(Q=Q, K=K, V=V if case["with_v"] else None, wq=wq if case["norm"] else None,
                wk=wk if case["norm"] else None, pos=pos, axes=axes,
                freq=freq.to(torch.float32).to(DEV))


def _mixture(H, n, d, mu, g):
    comp = torch.randint(0, mu.shape[1], (H, n), generator=g, device=DEV)
    x = torch.randn(H, n, d, generator=g, device=DEV)
    return (mu[torch.arange(H, device=DEV)[:, None], comp] + 0.3 * x).to(torch.bfloat16)


def _case_ranges(case):
    """[nq, 4] key ranges of a dense case, None without a mask."""
    if case["mask"] == "none":
        return None
    q, k, c = _lens(case["q"]), _lens(case["k"]), _lens(case["c"])
    prefix = int(case["prefix"]) if case["mask"] == "causal" else None
    return _numpy_ranges(q, k, c, prefix, case["pad"])


def _numpy_ranges(q, k, c, prefix, pad):
    rows = np.zeros((sum(q) + pad, 4), dtype=np.int64)
    qo, ko, co = _offsets(q), _offsets(k), _offsets(c)
    for b, n in enumerate(q):
        r = rows[qo[b]:qo[b + 1]]
        if len(k):
            r[:, 0], r[:, 1] = ko[b], ko[b + 1]
        if len(c):
            r[:, 2], r[:, 3] = co[b], co[b + 1]
            if prefix is not None:
                end = np.maximum(prefix, np.arange(1, n + 1) + c[b] - n)
                r[:, 3] = co[b] + np.clip(end, 0, c[b])
    return rows


def _dense_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    H, d = case["H"], case["d"]
    nq, nk, nc = sum(_lens(case["q"])) + case["pad"], sum(_lens(case["k"])), sum(_lens(case["c"]))
    mu = torch.randn(H, 32, d, generator=g, device=DEV)
    x = dict(Q=_mixture(H, nq, d, mu, g), K=_mixture(H, nk, d, mu, g),
             V=torch.randn(H, nk, d, generator=g, device=DEV).to(torch.bfloat16),
             Kc=None, Vc=None, ranges=None)
    if nc:
        x["Kc"] = _mixture(H, nc, d, mu, g)
        x["Vc"] = torch.randn(H, nc, d, generator=g, device=DEV).to(torch.bfloat16)
    r = _case_ranges(case)
    if r is not None:
        x["ranges"] = torch.from_numpy(r.astype(np.int32)).to(DEV)
    return x


def _ranges_inputs(case, seed):
    # the first segment's rows give some of theirs to the others: another seed, other offsets
    rng = np.random.default_rng(seed)

    def shuffled(text):
        lens = np.asarray(_lens(text), dtype=np.int64)
        if lens.size > 1:
            a, b = rng.integers(0, lens.size, 2)
            n = rng.integers(0, lens[a] + 1)
            lens[a] -= n
            lens[b] += n
        return [int(v) for v in lens]

    q, k = shuffled(case["q"]), shuffled(case["k"])
    c = q if case["c"] == case["q"] else shuffled(case["c"])
    n = len(q)
    prefix = None
    if case["prefix"]:
        prefix = [int(v) for v in rng.integers(0, int(case["prefix"]) + 1, n)]
    if n == 1:
        q = [max(1, q[0] - int(rng.integers(0, max(1, q[0] // 2))))]
    return q, k, c, prefix, sum(_lens(case["q"])) + case["pad"]


def prepare(case, seed):
    op = case["op"]
    state = dict(case=case)
    if op == "norm_rope":
        x = _rope_inputs(case, seed)
        H, N, d = x["Q"].shape
        for n in ("Q", "K", "V"):
            if x[n] is not None:
                x[n + "_out"] = torch.empty(H, N, d, dtype=x[n].dtype, device=DEV)
            else:
                x[n + "_out"] = None
    elif op == "ranges":
        q, k, c, prefix, nq = _ranges_inputs(case, seed)

        def put(v):
            return torch.tensor(v, dtype=torch.int32, device=DEV)

        x = dict(q=put(_offsets(q)), k=put(_offsets(k)) if k else None,
                 c=put(_offsets(c)) if c else None, nq=nq,
                 prefix=None if prefix is None else put(prefix),
                 ranges=torch.empty(nq, 4, dtype=torch.int32, device=DEV))
    else:
        x = _dense_inputs(case, seed)
        H, nq, d = x["Q"].shape
        x["out"] = torch.empty(H, nq, d, dtype=torch.bfloat16, device=DEV)
        x["lse"] = torch.empty(H, nq, dtype=torch.float32, device=DEV)
        if own:
            from block_sparse_attention_gather_b200 import spark_attend_dense_workspace_size
            nc = 0 if x["Kc"] is None else x["Kc"].shape[1]
            size = spark_attend_dense_workspace_size(H, nq, x["K"].shape[1], nc, d)
            x["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device=DEV)
    state.update(x)
    return state


# --------------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"norm_rope": _plain_norm_rope, "ranges": _plain_ranges,
            "dense": _plain_dense}[case["op"]](case, state)


def _run_own(case, s):
    import block_sparse_attention_gather_b200 as bsa
    if case["op"] == "norm_rope":
        outs = bsa.spark_qk_norm_rope(
            s["Q"], s["K"], s["V"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6,
            positions=s["pos"], inv_freq=s["freq"], axis_pairs=s["axes"],
            interleaved=case["layout"] == "interleaved", rope_scale=case["scale"],
            Q_out=s["Q_out"], K_out=s["K_out"], V_out=s["V_out"])
        return [t for t in outs if t is not None]
    if case["op"] == "ranges":
        return bsa.spark_attend_ranges(s["nq"], s["q"], s["k"], s["c"], prefix=s["prefix"],
                                       causal=case["causal"], ranges=s["ranges"])
    return bsa.spark_attend_dense(s["Q"], s["K"], s["V"], s["Kc"], s["Vc"], ranges=s["ranges"],
                                  out=s["out"], lse=s["lse"], workspace=s["ws"])


def _plain_norm_rope(case, s):
    angle = torch.cat([s["pos"][:, a:a + 1].double() * f.double()
                       for a, f in enumerate(s["freq"].split(s["axes"]))], dim=1)
    cos, sin = ((f(angle) * case["scale"]).float() for f in (torch.cos, torch.sin))
    r = 2 * cos.shape[1]

    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + 1e-6) * w
        t, rest = y[..., :r], y[..., r:]
        if case["layout"] == "half":
            a, b = t[..., :r // 2], t[..., r // 2:]
            t = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        else:
            a, b = t[..., 0::2], t[..., 1::2]
            t = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        return torch.cat([t, rest], dim=-1).to(x.dtype).contiguous()

    outs = [one(s["Q"], s["wq"]), one(s["K"], s["wk"])]
    if s["V"] is not None:
        outs.append(s["V"].contiguous())
    return outs


def _plain_ranges(case, s):
    qo = s["q"]
    i = torch.arange(s["nq"], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(qo[1:].contiguous(), i, right=True)
    live = b < qo.numel() - 1
    b = b.clamp(max=qo.numel() - 2)
    out = torch.zeros(s["nq"], 4, dtype=torch.int32, device=DEV)
    if s["k"] is not None:
        out[:, 0], out[:, 1] = s["k"][b], s["k"][b + 1]
    if s["c"] is not None:
        c0, c1 = s["c"][b], s["c"][b + 1]
        if case["causal"]:
            end = i - qo[b] + 1 + (c1 - c0) - (qo[b + 1] - qo[b])
            if s["prefix"] is not None:
                end = torch.maximum(end, s["prefix"][b])
            c1 = c0 + torch.minimum(end.clamp(min=0), c1 - c0)
        out[:, 2], out[:, 3] = c0, c1
    return out * live[:, None].to(torch.int32)


def _plain_dense(case, s):
    Q, K, V, Kc, Vc = s["Q"], s["K"], s["V"], s["Kc"], s["Vc"]
    H, nq, d = Q.shape
    nk = K.shape[1]
    n = nk + (0 if Kc is None else Kc.shape[1])
    out = torch.empty(H, nq, d, dtype=Q.dtype, device=DEV)
    lse = torch.empty(H, nq, dtype=torch.float32, device=DEV)
    step = max(1, (1 << 28) // n)
    j = torch.arange(n, device=DEV)
    for h in range(H):
        k, v = K[h].float(), V[h].float()
        if Kc is not None:
            k, v = torch.cat([k, Kc[h].float()]), torch.cat([v, Vc[h].float()])
        for a in range(0, nq, step):
            S = (Q[h, a:a + step].float() @ k.T) * (1.0 / math.sqrt(d))
            if s["ranges"] is not None:
                r = s["ranges"][a:a + step, :, None]
                video = (j >= r[:, 0]) & (j < r[:, 1]) & (j < nk)
                context = (j >= r[:, 2] + nk) & (j < r[:, 3] + nk)
                S = S.masked_fill(~(video | context), -math.inf)
            m = S.amax(dim=1, keepdim=True)
            p = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
            l = p.sum(dim=1, keepdim=True)
            o = (p @ v) / torch.where(l == 0, torch.ones_like(l), l)
            out[h, a:a + step] = o.to(out.dtype)
            lse[h, a:a + step] = (m + torch.log(l))[:, 0]
    return out, lse


# ------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "norm_rope":
        H, N, d = case["H"], case["N"], case["d"]
        size = 2 if case["dtype"] == "bf16" else 4
        axes = [int(a) for a in case["axes"].split(",")]
        tensors = 3 if case["with_v"] else 2
        return {"bytes": 2 * tensors * H * N * d * size + 4 * N * len(axes) + 4 * sum(axes)
                + (8 * d if case["norm"] else 0), "flops": 2 * H * N * 6 * d}
    q, k, c = _lens(case["q"]), _lens(case["k"]), _lens(case["c"])
    nq = sum(q) + case["pad"]
    if case["op"] == "ranges":
        return {"bytes": 16 * nq + 4 * (len(q) + 1 + (len(k) + 1 if k else 0)
                                        + (len(c) + 1 if c else 0)
                                        + (len(q) if case["prefix"] else 0)), "flops": 0}
    H, d = case["H"], case["d"]
    r = _case_ranges(case)
    if r is None:
        pairs, keys = nq * (sum(k) + sum(c)), sum(k) + sum(c)
    else:
        pairs = int((r[:, 1] - r[:, 0]).sum() + (r[:, 3] - r[:, 2]).sum())
        keys = 0
        for lo, hi, n in ((r[:, 0], r[:, 1], sum(k)), (r[:, 2], r[:, 3], sum(c))):
            edge = np.zeros(n + 1, dtype=np.int64)
            live = hi > lo
            np.add.at(edge, lo[live], 1)
            np.add.at(edge, hi[live], -1)
            keys += int((np.cumsum(edge)[:n] > 0).sum())
    return {"bytes": H * (2 * nq * d * 2 + 2 * keys * d * 2 + 4 * nq) + (16 * nq if r is not None
                                                                         else 0),
            "flops": 4 * H * pairs * d}


# ------------------------------------------------------------------------------------ exact

def exact(case, seed):
    """The operator's definition in 64 bits on the inputs of `seed`."""
    if case["op"] == "norm_rope":
        return _exact_norm_rope(case, _rope_inputs(case, seed))
    if case["op"] == "ranges":
        return _exact_ranges(case, seed)
    return _exact_dense(case, _dense_inputs(case, seed))


def _exact_norm_rope(case, x):
    turn = []
    at = 0
    for a, n in enumerate(x["axes"]):
        turn.append(torch.outer(x["pos"][:, a].double(), x["freq"][at:at + n].double()))
        at += n
    turn = torch.cat(turn, dim=1)
    unit = torch.polar(torch.full_like(turn, case["scale"]), turn)           # [N, pairs]
    outs = []
    for t, w in ((x["Q"], x["wq"]), (x["K"], x["wk"])):
        y = t.double()
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + 1e-6) * w.double()
        y = y.contiguous()
        if case["layout"] == "half":
            z = torch.complex(y[..., :at], y[..., at:2 * at]) * unit
            y[..., :at], y[..., at:2 * at] = z.real, z.imag
        else:
            z = torch.view_as_complex(y[..., :2 * at].reshape(*y.shape[:-1], at, 2)) * unit
            y[..., :2 * at] = torch.view_as_real(z).flatten(-2)
        outs.append(y)
    if x["V"] is not None:
        outs.append(x["V"].double().contiguous())
    return outs


def _exact_ranges(case, seed):
    q, k, c, prefix, nq = _ranges_inputs(case, seed)
    rows = np.zeros((nq, 4), dtype=np.int32)
    qo, ko, co = _offsets(q), _offsets(k), _offsets(c)
    i = 0
    for b in range(len(q)):
        for n in range(q[b]):
            lo, hi = (ko[b], ko[b + 1]) if k else (0, 0)
            clo, chi = (co[b], co[b + 1]) if c else (0, 0)
            if c and case["causal"]:
                seen = max(n + 1 + c[b] - q[b], prefix[b] if prefix else 0)
                chi = clo + min(max(seen, 0), c[b])
            rows[i] = (lo, hi, clo, chi)
            i += 1
    return torch.from_numpy(rows)


def _exact_dense(case, x):
    H, nq, d = x["Q"].shape
    nk = x["K"].shape[1]
    keys = x["K"] if x["Kc"] is None else torch.cat([x["K"], x["Kc"]], dim=1)
    values = x["V"] if x["Vc"] is None else torch.cat([x["V"], x["Vc"]], dim=1)
    n = keys.shape[1]
    out = torch.zeros(H, nq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(H, nq, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // n)
    index = torch.arange(n, device=DEV)[None, :]
    for h in range(H):
        kt, v = keys[h].double().T.contiguous(), values[h].double()
        for a in range(0, nq, step):
            z = torch.mm(x["Q"][h, a:a + step].double(), kt).div_(math.sqrt(d))
            if x["ranges"] is not None:
                r = x["ranges"][a:a + step].long()
                dead = torch.where(index < nk,
                                   (index < r[:, 0:1]) | (index >= r[:, 1:2]),
                                   (index < r[:, 2:3] + nk) | (index >= r[:, 3:4] + nk))
                z[dead] = -math.inf
            e = torch.logsumexp(z, dim=1)
            lse[h, a:a + step] = e
            z.sub_(e.masked_fill(e == -math.inf, 0.0)[:, None]).exp_()
            out[h, a:a + step] = z @ v
    return out, lse
