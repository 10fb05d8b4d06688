"""What is measured of the operators around the experts of a mixture-of-experts layer, and their plain forms.

    grouped_mm      y_r  = W_e x_r                      rows r of expert e's segment
    grouped_dgrad   dx_r = W_e^T dy_r                   its gradient for the rows
    grouped_wgrad   dW_e = sum_{r in e} dy_r x_r^T      its gradient for the weights
    grouped_lora    y_r  = W_e x_r + s_a B_{a,e} (A_{a,e} x_r)      a = the row's adapter, -1 for none
    clip_grads      n = sqrt(sum_i |g_i|^2),  out_i = g_i min(1, max_norm / (n + eps))

Segment e holds the rows [offsets[e], offsets[e] + counts[e]); without counts it ends where the next one
starts.  The sizes are those of this repository's workloads (d = 4096, ffn = 14336, 8 experts, top-2),
of its small test layers, and odd ones between.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's two experts, up projection: all latency and weight streaming
        dict(name="mm-token", op="grouped_mm", M=2, E=8, N=14336, K=4096, dtype="bf16", out="bf16", skew=0.0, align=1,
             split=1),
        # a decode batch of 16 tokens, down projection into the fp32 rows that a combine reads
        dict(name="mm-decode", op="grouped_mm", M=32, E=8, N=4096, K=14336, dtype="bf16", out="f32", skew=0.3, align=1,
             split=2),
        # a 4096-token prefill on the padded segments that moe_dispatch lays out
        dict(name="mm-prefill", op="grouped_mm", M=8192, E=8, N=14336, K=4096, dtype="bf16", out="bf16", skew=0.2,
             align=128, split=3),
        # a small fp32 layer of odd sizes
        dict(name="dgrad-odd-f32", op="grouped_dgrad", M=1003, E=5, N=1416, K=520, dtype="f32", out="f32", skew=0.8,
             align=1, split=4),
        # a 4096-token training step, gradient of the rows
        dict(name="dgrad-train", op="grouped_dgrad", M=8192, E=8, N=14336, K=4096, dtype="bf16", out="bf16", skew=0.2,
             align=1, split=5),
        # many small experts with few and uneven rows, some without any
        dict(name="wgrad-odd", op="grouped_wgrad", M=1531, E=32, N=776, K=1288, dtype="bf16", out="bf16", skew=1.2,
             align=1, split=6),
        # a 4096-token training step, gradient of the weights in fp32
        dict(name="wgrad-train", op="grouped_wgrad", M=8192, E=8, N=14336, K=4096, dtype="bf16", out="f32", skew=0.2,
             align=1, split=7),
        # a decode batch whose 16 tokens belong to many requests with an adapter each
        dict(name="lora-decode", op="grouped_lora", M=32, E=8, N=14336, K=4096, L=16, R=16, run=1, out="bf16",
             skew=0.3, split=8),
        # a mixed batch on one shared projection: decode tokens and short prompts
        dict(name="lora-shared", op="grouped_lora", M=205, E=1, N=4096, K=4096, L=40, R=32, run=6, out="bf16",
             skew=0.0, split=9),
        # a prefill batch of long prompts, an adapter to each
        dict(name="lora-prefill", op="grouped_lora", M=4096, E=8, N=14336, K=4096, L=12, R=64, run=90, out="bf16",
             skew=0.2, split=10),
        # the gradients of a two-layer model of the tests' size, router gradients in fp32
        dict(name="clip-small", op="clip_grads", layers=2, E=8, d=256, F=512, mixed=True, extra=7, max_norm=1.0),
        # one full layer's gradients, rounded to bf16 by the backward
        dict(name="clip-layer", op="clip_grads", layers=1, E=8, d=4096, F=14336, mixed=False, extra=1, max_norm=1.0),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["grouped_mm", "grouped_mm", "grouped_dgrad", "grouped_wgrad", "grouped_lora", "grouped_lora",
                     "clip_grads"])
    if op == "clip_grads":
        while True:
            c = dict(op=op, layers=rng.randint(1, 8), E=_log_int(rng, 1, 32), d=_log_int(rng, 64, 4096, 8),
                     F=_log_int(rng, 128, 14336, 8), mixed=rng.random() < 0.5, extra=rng.randint(0, 20),
                     max_norm=rng.choice([0.5, 1.0, 1e4]))
            if c["layers"] * c["E"] * c["d"] * c["F"] <= 2.0e8:
                return c
    while True:
        c = dict(op=op, M=_log_int(rng, 1, 8192), E=_log_int(rng, 1, 32), N=_log_int(rng, 64, 14336, 8),
                 K=_log_int(rng, 64, 14336, 8), skew=rng.choice([0.0, 0.3, 1.5]), split=rng.randint(0, 1 << 30))
        if c["M"] * c["N"] * c["K"] > 4.0e11 or c["E"] * c["N"] * c["K"] > 4.5e8:
            continue
        if op == "grouped_lora":
            c.update(L=_log_int(rng, 1, 64), R=rng.choice([8, 16, 24, 32, 64, 128]), run=_log_int(rng, 1, 200),
                     out=rng.choice(["bf16", "f32"]))
            if c["L"] * c["E"] * c["R"] * (c["N"] + c["K"]) > 4.0e8:
                continue
        else:
            c.update(dtype=rng.choice(["bf16", "bf16", "f32"]), align=rng.choice([1, 1, 128]))
            c["out"] = "f32" if c["dtype"] == "f32" else rng.choice(["bf16", "f32"])
            if c["dtype"] == "f32" and c["M"] * c["N"] * c["K"] > 2.0e10:
                continue
        return c


def _counts(case):
    """Rows of each expert: M assignments drawn with uneven popularity, the same for every seed."""
    rng = np.random.default_rng(case["split"])
    p = np.exp(case["skew"] * rng.standard_normal(case["E"]))
    return rng.multinomial(case["M"], p / p.sum()).tolist()


def _segments(case):
    """(start, rows) of each expert and the number of rows of the buffers."""
    align = case.get("align", 1)
    segs, row = [], 0
    for n in _counts(case):
        segs.append((row, n))
        row += -(-n // align) * align
    return segs, row


def _adapters(case):
    """The adapter of each row: requests are runs of rows of `run` on average, one in eight without an adapter."""
    rng = random.Random(case["split"] + 1)
    ids = []
    while len(ids) < case["M"]:
        n = 1 if case["run"] == 1 else rng.randint(1, 2 * case["run"] - 1)
        a = -1 if rng.random() < 0.125 else rng.randrange(case["L"])
        ids += [a] * n
    return ids[:case["M"]]


def _pairs(case):
    """(adapter, expert) -> rows, for the pairs that occur."""
    ids = _adapters(case)
    pairs = {}
    for e, (start, n) in enumerate(_segments(case)[0]):
        for r in range(start, start + n):
            if ids[r] >= 0:
                pairs.setdefault((ids[r], e), []).append(r)
    return pairs


def _grad_shapes(case):
    """(shape, dtype) of every gradient: per layer dWg, dW1, dW3, dW2 and the norm's gain, then odd-sized others."""
    E, d, F = case["E"], case["d"], case["F"]
    big = torch.bfloat16
    out = []
    for layer in range(case["layers"]):
        w = torch.float32 if case["mixed"] and layer % 2 else big
        out += [((E, d), torch.float32), ((E, F, d), w), ((E, F, d), w), ((E, d, F), w), ((d,), torch.float32)]
    rng = random.Random(case["extra"])
    for i in range(case["extra"]):
        out.append(((rng.randint(1, 4000),), torch.float32 if i % 2 else big))
    return out


# ------------------------------------------------------------------ state

def _randn(gen, shape, scale, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "clip_grads":
        grads = []
        for i, (shape, dtype) in enumerate(_grad_shapes(case)):
            # gradients differ in size from tensor to tensor by orders of magnitude
            grads.append(_randn(gen, shape, 1e-3 * math.exp(0.7 * ((7 * i) % 5 - 2)), dtype))
        return dict(case=case, grads=grads, out=[torch.empty_like(g) for g in grads])
    M, E, N, K, op = case["M"], case["E"], case["N"], case["K"], case["op"]
    segs, rows = _segments(case)
    dtype = DTYPES[case.get("dtype", "bf16")]
    starts = [s for s, _ in segs] + [rows]
    st = dict(case=case, segs=segs)
    st["offsets"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    # packed rows: the offsets say it all; padded segments come with their counts, as from a dispatch
    st["counts"] = (torch.tensor([n for _, n in segs], dtype=torch.int32, device="cuda")
                    if case.get("align", 1) > 1 else None)
    odt = DTYPES[case["out"]]
    if op != "grouped_dgrad":
        st["x"] = _randn(gen, (rows, K), 1.0, dtype)
    if op in ("grouped_dgrad", "grouped_wgrad"):
        st["dy"] = _randn(gen, (rows, N), 1e-2, dtype)
    if op != "grouped_wgrad":
        st["W"] = torch.empty((E, N, K), dtype=dtype, device="cuda")
        for e in range(E):
            st["W"][e] = _randn(gen, (N, K), 1.0 / math.sqrt(K), dtype)
    shape = {"grouped_dgrad": (rows, K), "grouped_wgrad": (E, N, K)}.get(op, (rows, N))
    st["out"] = torch.zeros(shape, dtype=odt, device="cuda")
    if op == "grouped_lora":
        L, R = case["L"], case["R"]
        st["A"] = torch.empty((L, E, R, K), dtype=dtype, device="cuda")
        st["B"] = torch.empty((L, E, N, R), dtype=dtype, device="cuda")
        for a in range(L):
            st["A"][a] = _randn(gen, (E, R, K), 1.0 / math.sqrt(K), dtype)
            st["B"][a] = _randn(gen, (E, N, R), 0.5 / math.sqrt(R), dtype)
        st["scale"] = torch.rand(L, generator=gen, device="cuda", dtype=torch.float32) + 0.5
        st["adapter"] = torch.tensor(_adapters(case), dtype=torch.int32, device="cuda")
        st["pairs"] = {p: torch.tensor(r, device="cuda") for p, r in _pairs(case).items()}
    return st


# ------------------------------------------------------------------ one pass

def _run_own(st):
    import sparse_mixture_experts_14_b200 as moe
    op = st["case"]["op"]
    if op == "clip_grads":
        return moe.moe_clip_grads(st["grads"], st["case"]["max_norm"], eps=EPS, out=st["out"])
    seg = dict(counts=st["counts"], out=st["out"])
    if op == "grouped_mm":
        return moe.moe_grouped_mm(st["x"], st["W"], st["offsets"], **seg)
    if op == "grouped_dgrad":
        return moe.moe_grouped_dgrad(st["dy"], st["W"], st["offsets"], **seg)
    if op == "grouped_wgrad":
        return moe.moe_grouped_wgrad(st["dy"], st["x"], st["offsets"], **seg)
    return moe.moe_grouped_lora(st["x"], st["W"], st["offsets"], st["A"], st["B"], st["scale"], st["adapter"],
                                out=st["out"])


def run(st):
    if own:
        return _run_own(st)
    case, op = st["case"], st["case"]["op"]
    if op == "clip_grads":
        # squares summed in 64 bits: a sum over 1e9 terms
        sq = torch.stack([(g.float() ** 2).sum(dtype=torch.float64) for g in st["grads"]]).sum()
        norm = sq.sqrt()
        coef = torch.clamp(case["max_norm"] / (norm + EPS), max=1.0).float()
        for g, o in zip(st["grads"], st["out"]):
            o.copy_(g.float() * coef)
        return norm.float().reshape(1), st["out"]
    out = st["out"]
    for e, (s, n) in enumerate(st["segs"]):
        if op == "grouped_wgrad":
            out[e] = (st["dy"][s:s + n].float().t() @ st["x"][s:s + n].float()).to(out.dtype)
        elif n == 0:
            continue
        elif op == "grouped_dgrad":
            out[s:s + n] = (st["dy"][s:s + n].float() @ st["W"][e].float()).to(out.dtype)
        else:
            y = st["x"][s:s + n].float() @ st["W"][e].float().t()
            if op == "grouped_lora":
                for (a, ea), rows in st["pairs"].items():
                    if ea == e:
                        u = st["x"][rows].float() @ st["A"][a, e].float().t()
                        y.index_add_(0, rows - s, (u * st["scale"][a]) @ st["B"][a, e].float().t())
            out[s:s + n] = y.to(out.dtype)
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "clip_grads":
        n, b = 0, 4
        for shape, dtype in _grad_shapes(case):
            k = math.prod(shape)
            n += k
            b += 2 * k * (2 if dtype == torch.bfloat16 else 4)
        return {"bytes": b, "flops": 3 * n}
    M, E, N, K, op = case["M"], case["E"], case["N"], case["K"], case["op"]
    es = 2 if case.get("dtype", "bf16") == "bf16" else 4
    os_ = 2 if case["out"] == "bf16" else 4
    used = sum(1 for n in _counts(case) if n)
    if op == "grouped_wgrad":
        return {"bytes": M * (N + K) * es + E * N * K * os_, "flops": 2 * M * N * K}
    rows_in, rows_out = (N, K) if op == "grouped_dgrad" else (K, N)
    b = M * rows_in * es + M * rows_out * os_ + used * N * K * es + 4 * (E + 1)
    f = 2 * M * N * K
    if op == "grouped_lora":
        pairs = _pairs(case)
        b += len(pairs) * case["R"] * (N + K) * es + 4 * M
        f += 2 * sum(len(r) for r in pairs.values()) * case["R"] * (N + K)
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64
    if case["op"] == "clip_grads":
        total = 0.0
        for g in st["grads"]:
            total += torch.dot(g.reshape(-1).to(D), g.reshape(-1).to(D)).item()
        n = math.sqrt(total)
        c = min(1.0, case["max_norm"] / (n + EPS))
        return torch.tensor([n], dtype=D, device="cuda"), [g.to(D) * c for g in st["grads"]]
    out = torch.zeros(st["out"].shape, dtype=D, device="cuda")
    off = st["offsets"].tolist()
    cnt = st["counts"].tolist() if st["counts"] is not None else [b - a for a, b in zip(off, off[1:])]
    ids = st["adapter"].tolist() if "adapter" in st else None
    for e in range(case["E"]):
        r = slice(off[e], off[e] + cnt[e])
        if cnt[e] == 0:
            continue
        if case["op"] == "grouped_wgrad":
            out[e] = torch.einsum("rn,rk->nk", st["dy"][r].to(D), st["x"][r].to(D))
        elif case["op"] == "grouped_dgrad":
            out[r] = torch.einsum("rn,nk->rk", st["dy"][r].to(D), st["W"][e].to(D))
        else:
            out[r] = torch.einsum("rk,nk->rn", st["x"][r].to(D), st["W"][e].to(D))
            for a in sorted({i for i in (ids[r] if ids else []) if i >= 0}):
                mine = [i for i in range(r.start, r.stop) if ids[i] == a]
                low = torch.einsum("rk,jk->rj", st["x"][mine].to(D), st["A"][a, e].to(D))
                out[mine] += st["scale"][a].to(D) * torch.einsum("rj,nj->rn", low, st["B"][a, e].to(D))
    return out
