"""The library's scored router and its microscaled 4-bit (MXFP4) operators, as cases that can be timed and compared.

Four operators:

* ``route``    moe_route_scored: softmax or sigmoid scores, a balance bias, expert groups, top-k, renormalised weights
* ``quantize`` moe_mx_quantize and moe_mx_dequantize: rows (each written to its experts' places, or as they are) to MXFP4 and back to values
* ``product``  moe_mx_grouped_gemm: rows in MXFP4 against expert matrices in MXFP4
* ``ffn``      moe_mx_quantize and moe_grouped_ffn_mx: an expert SwiGLU FFN from bf16 tokens to permuted outputs

MXFP4: 4-bit e2m1 elements (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives, two to a byte, the even element in the low
nibble), one power-of-two scale (a byte, exponent + 127) for each 32 elements along K.  A weight matrix [N][K] is its
codes [N][K / 2], then its scales in tiles of 128 rows x 128 K (512 bytes: row r of a tile, block b at
(r % 32) * 16 + r / 32 * 4 + b), tile rows in order, K inside.  An expert's FFN blob is the matrix of its gate and up rows
(32 gate rows, 32 up rows, 32 gate rows, ...) and then its down matrix.
"""
import math

import torch

own = False

GATE_STD = 0.02   # router and expert weights ~ N(0, 0.02^2), activations ~ N(0, 1): the workloads' distributions


def listed():
    return [
        # one token of a decode step: a 64-expert layer of hidden size 2048, sigmoid scores with a balance bias in 8 groups
        dict(name="route decode 1", op="route", T=1, d=2048, E=64, k=8, scoring="sigmoid", bias=True, groups=8, kept=4,
             group_top=2, renorm=True, scale=2.5),
        # a chunk of a prompt through a softmax router without bias or groups, probabilities as they are
        dict(name="route chunk 250", op="route", T=250, d=4096, E=128, k=8, scoring="softmax", bias=False, groups=1,
             kept=1, group_top=1, renorm=False, scale=1.0),
        # a whole prefill batch of the 4096-token workload, many experts in groups
        dict(name="route prefill 4096", op="route", T=4096, d=2048, E=256, k=8, scoring="sigmoid", bias=True, groups=8,
             kept=4, group_top=2, renorm=True, scale=2.5),
        # the largest batch, an odd number of tokens, wide rows
        dict(name="route prefill 8191", op="route", T=8191, d=4096, E=256, k=8, scoring="sigmoid", bias=True, groups=1,
             kept=1, group_top=1, renorm=True, scale=1.0),
        # the rows of one decode step's 8 tokens, each for its 8 experts
        dict(name="quantize decode 8", op="quantize", T=8, K=2048, k=8, dtype="bf16"),
        # the activations of the 4096-token prefill, in expert order
        dict(name="quantize gather 4096", op="quantize", T=4096, K=2048, k=8, dtype="bf16"),
        # fp32 rows as they are (weights, or a checkpoint's tensor), an odd number of them
        dict(name="quantize fp32 28673", op="quantize", T=28673, K=4096, k=0, dtype="fp32"),
        # a decode step's rows through one matrix of 64 experts, most of them with a row or two
        dict(name="product decode 16", op="product", T=16, E=64, k=8, N=2048, K=1024, out="fp16"),
        # one dense matrix (a shared expert) on a prefill batch of odd length
        dict(name="product dense 4095", op="product", T=4095, E=1, k=1, N=4096, K=4096, out="bf16"),
        # the expert FFN of one decode token, of a small batch, and of the largest prefill of wide experts
        dict(name="ffn decode 1", op="ffn", T=1, E=64, k=8, d=2048, F=1024),
        dict(name="ffn prefill 4096", op="ffn", T=4096, E=64, k=8, d=2048, F=1024),
        dict(name="ffn wide 8192", op="ffn", T=8192, E=8, k=2, d=4096, F=14336),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "quantize", "product", "ffn"])
    if op == "route":
        E = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256])
        G = rng.choice([g for g in (1, 2, 4, 8) if E % g == 0 and E // g >= 4])
        kept = rng.randint(max(1, G // 2), G)
        k = rng.randint(1, min(8, kept * (E // G)))
        return dict(op=op, T=_log_int(rng, 1, 8191), d=32 * rng.randint(8, 128), E=E, k=k,
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=G, kept=kept,
                    group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    if op == "quantize":
        k = rng.choice([0, 1, 2, 4, 8])
        return dict(op=op, T=_log_int(rng, 1, 4096 if k else 28673), K=32 * rng.randint(4, 128 if not k else 64), k=k,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    E = rng.choice([1, 4, 8, 16, 64])
    k = rng.randint(1, min(8, E))
    if op == "product":
        return dict(op=op, T=_log_int(rng, 1, 4095), E=E, k=k, N=128 * rng.randint(2, 16), K=128 * rng.randint(2, 16),
                    out=rng.choice(["fp16", "bf16", "fp32"]))
    return dict(op=op, T=_log_int(rng, 1, 4096), E=E, k=k, d=128 * rng.randint(2, 32), F=128 * rng.randint(2, 12))


# ---- inputs -------------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(v):
    """MXFP4 codes (one element a byte) and scale bytes of fp32 values [..., K]."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    a = b.abs().amax(-1)
    e = torch.where(a > 0, (torch.frexp(a)[1] - 3).clamp(-127, 127), torch.full_like(a, -127).int())
    m = b.abs() * _pow2(-e).unsqueeze(-1)
    half = torch.round(m * 2)                    # steps of 0.5 below 2, of 1 below 4, of 2 above
    code = torch.where(m < 2, half, torch.where(m < 4, 2 + torch.round(m), torch.clamp(4 + torch.round(m * 0.5), max=7)))
    code = (code + 8 * torch.signbit(b)).to(torch.uint8).reshape(v.shape)
    return code, (e + 127).to(torch.uint8)


def _matrix(w):
    """fp32 [N][K] -> the bytes of an MXFP4 matrix."""
    N, K = w.shape
    c, s = _codes(w)
    c = c.view(N, K // 2, 2)
    packed = c[..., 0] | (c[..., 1] << 4)
    s = s.view(N // 128, 4, 32, K // 128, 4).permute(0, 3, 2, 1, 4)
    return torch.cat([packed.reshape(-1), s.reshape(-1)])


def _routing(case, gen):
    """Distinct random experts for each token, rows sorted by expert: perm, offsets, the experts with rows, the longest run."""
    T, E, k = case["T"], case["E"], case["k"]
    ids = torch.rand(T, E, generator=gen, device="cuda").argsort(-1)[:, :k].reshape(-1)
    perm = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return perm.int(), offsets, counts.nonzero().reshape(-1), int(counts.max())


def _inverse(perm):
    inv = torch.empty_like(perm)
    inv[perm.long()] = torch.arange(perm.numel(), dtype=torch.int32, device=perm.device)
    return inv


_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    op, T = case["op"], case["T"]
    if op == "route":
        s["x"] = normal(T, case["d"]).bfloat16()
        s["w"] = normal(case["E"], case["d"], std=GATE_STD)
        s["bias"] = normal(case["E"], std=0.05) if case["bias"] else None
    elif op == "quantize":
        # magnitudes over a few octaves from row to row, as hidden states have them
        s["x"] = (normal(T, case["K"]) * torch.exp2(normal(T, 1))).to(_DTYPES[case["dtype"]])
        s["perm"] = torch.randperm(T * case["k"], generator=g, device="cuda").int() if case["k"] else None
        s["inv_perm"] = _inverse(s["perm"]) if case["k"] else None
    elif op == "product":
        s["perm"], s["offsets"], s["active"], s["cap"] = _routing(case, g)
        N, K = case["N"], case["K"]
        c, s["scales"] = _codes(normal(T * case["k"], K))
        s["codes"] = c[:, 0::2] | (c[:, 1::2] << 4)
        s["mats"] = torch.stack([_matrix(normal(N, K, std=GATE_STD)) for _ in range(case["E"])])
    else:
        s["perm"], s["offsets"], s["active"], s["cap"] = _routing(case, g)
        s["inv_perm"] = _inverse(s["perm"])
        d, F = case["d"], case["F"]
        s["x"] = normal(T, d).bfloat16()
        blobs = []
        for _ in range(case["E"]):
            # 32 gate rows, 32 up rows, and so on: independent draws of one distribution
            blobs.append(torch.cat([_matrix(normal(2 * F, d, std=GATE_STD)), _matrix(normal(d, F, std=GATE_STD))]))
        s["blobs"] = torch.stack(blobs)
    return s


# ---- the plain form -----------------------------------------------------------------------------------------------

def _pow2(e):
    """2^e, exactly, as fp32 (e a whole-numbered tensor in [-148, 127])."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64).to(torch.float32)


def _values(codes, scales):
    """fp32 values [..., K] of packed codes [..., K/2] and scale bytes [..., K/32]."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    mag = n & 7
    e = (mag >> 1).int()
    f = (mag & 1).float()
    v = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * _pow2(e - 1))
    v = torch.where(n >= 8, -v, v)
    v = v.reshape(*v.shape[:-1], -1, 32) * _pow2(scales.int() - 127).unsqueeze(-1)
    return v.flatten(-2)


def _rounded(v):
    """fp32 [..., K] -> the values that its MXFP4 form stands for."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    a = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(a)[1] - 3).clamp(-127, 127)
    m = b.abs() * _pow2(-e)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(m / step) * step, max=6.0) * _pow2(e)
    return torch.where(b < 0, -q, q).reshape(v.shape)


def _matrix_values(raw, N, K):
    """fp32 [n][N][K] of the bytes [n][...] of MXFP4 matrices."""
    n = raw.shape[0]
    codes = raw[:, :N * K // 2].reshape(n, N, K // 2)
    s = raw[:, N * K // 2:].reshape(n, N // 128, K // 128, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(n, N, K // 32)
    return _values(codes, s)


def _grouped(s, rows, weights):
    """rows [R][K] in expert order times the active experts' weights [A][N][K]: the rows of each expert laid side by side."""
    starts = s["offsets"][s["active"]].long()
    ends = s["offsets"][s["active"] + 1].long()
    p = torch.arange(rows.shape[0], device=rows.device)
    a = torch.searchsorted(ends, p, right=True)
    at = p - starts[a]
    side = rows.new_zeros(weights.shape[0], s["cap"], rows.shape[1])
    side[a, at] = rows
    return torch.matmul(side, weights.transpose(1, 2))[a, at]


def _choice(case, logits, bias):
    """The chosen experts, and the scores of all, from logits in 64 bits."""
    scores = torch.sigmoid(logits) if case["scoring"] == "sigmoid" else torch.softmax(logits, -1)
    c = scores if bias is None else scores + bias.double()
    if case["groups"] > 1:
        T, G = c.shape[0], case["groups"]
        by = c.view(T, G, -1)
        top = by.sort(dim=-1, descending=True)[0][..., :case["group_top"]].sum(-1)
        kept = top.sort(dim=-1, descending=True, stable=True)[1][:, :case["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=c.device)
        keep[torch.arange(T, device=c.device)[:, None], kept] = True
        c = torch.where(keep[..., None], by, torch.full_like(by, -math.inf)).view(T, -1)
    return c.sort(dim=-1, descending=True, stable=True)[1][:, :case["k"]], scores


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state, case, op)
    if op == "route":
        # in 64 bits: the choice between two experts turns on their scores' last digits
        logits = state["x"].double() @ state["w"].double().t()
        idx, scores = _choice(case, logits, state["bias"])
        w = scores.gather(1, idx)
        if case["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        return {"idx": idx.int(), "w": (w * case["scale"]).float()}
    if op == "quantize":
        x = state["x"].float()
        if state["perm"] is not None:
            x = x[(state["perm"] // case["k"]).long()]
        return _rounded(x).bfloat16()
    if op == "product":
        rows = _values(state["codes"], state["scales"])
        w = _matrix_values(state["mats"][state["active"]], case["N"], case["K"])
        return _grouped(state, rows, w).to(_DTYPES[case["out"]])
    d, F = case["d"], case["F"]
    rows = _rounded(state["x"].float())[(state["perm"] // case["k"]).long()]
    raw = state["blobs"][state["active"]]
    split = F * d + F * d // 16                    # bytes of the gate and up matrix
    gu = _grouped(state, rows, _matrix_values(raw[:, :split], 2 * F, d)).view(-1, F // 32, 2, 32)
    gate, up = gu[:, :, 0].reshape(-1, F), gu[:, :, 1].reshape(-1, F)
    h = gate * torch.sigmoid(gate) * up
    return _grouped(state, _rounded(h), _matrix_values(raw[:, split:], d, F)).half()


# ---- the framework's calls ----------------------------------------------------------------------------------------

def _run_own(state, case, op):
    from quantized_moe_expert_histogram_b200 import moeq
    if op == "route":
        idx, w = moeq.moe_route_scored(
            state["x"], state["w"], case["k"], scoring=case["scoring"], bias=state["bias"], n_groups=case["groups"],
            topk_groups=case["kept"], group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
        return {"idx": idx, "w": w}
    if op == "quantize":
        codes, scales = moeq.moe_mx_quantize(state["x"], inv_perm=state["inv_perm"], k=max(1, case["k"]))
        return moeq.moe_mx_dequantize(codes, scales, dtype=torch.bfloat16)
    if op == "product":
        return moeq.moe_mx_grouped_gemm(state["codes"], state["scales"], state["offsets"], state["mats"], case["N"],
                                        dtype=_DTYPES[case["out"]])
    codes, scales = moeq.moe_mx_quantize(state["x"], inv_perm=state["inv_perm"], k=case["k"])
    return moeq.moe_grouped_ffn_mx(codes, scales, state["offsets"], state["blobs"], case["F"])


# ---- what a pass cannot do without --------------------------------------------------------------------------------

def work(case):
    op, T, k = case["op"], case["T"], case["k"]
    mx = 0.5 + 1 / 32                              # bytes an MXFP4 element takes
    if op == "route":
        return {"bytes": 2.0 * T * case["d"] + 4.0 * case["E"] * (case["d"] + 1) + 8.0 * T * k,
                "flops": 2.0 * T * case["E"] * case["d"]}
    if op == "quantize":
        size = 4 if case["dtype"] == "fp32" else 2
        rows = T * max(1, k)
        return {"bytes": T * case["K"] * size + 4.0 * rows * (k > 0) + rows * case["K"] * (mx + 2.0), "flops": 4.0 * rows * case["K"]}
    E, rows = case["E"], T * k
    active = E * (1 - (1 - k / E) ** T)            # experts that have a row, on average
    if op == "product":
        N, K = case["N"], case["K"]
        return {"bytes": active * N * K * mx + rows * K * mx + rows * N * (4.0 if case["out"] == "fp32" else 2.0),
                "flops": 2.0 * rows * N * K}
    d, F = case["d"], case["F"]
    return {"bytes": active * 3 * d * F * mx + 2.0 * T * d + 2.0 * rows * d, "flops": 6.0 * rows * d * F}


# ---- the definition in 64 bits, expert by expert and pick by pick --------------------------------------------------

_TABLE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _nearest(v):
    """MXFP4 values of v (64 bits): each element the nearest grid point, of two equally near the one with the even code."""
    K = v.shape[-1]
    b = v.reshape(-1, 32)
    out = torch.empty_like(b)
    grid = torch.tensor(_TABLE[:8], dtype=torch.float64, device=v.device)
    for at in range(0, b.shape[0], 1 << 20):
        c = b[at:at + (1 << 20)]
        a = c.abs().amax(1)
        e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
        e = torch.where(torch.exp2(e) > a, e - 1, torch.where(torch.exp2(e + 1) <= a, e + 1, e)) - 2
        unit = torch.exp2(e.clamp(-127, 127))[:, None]
        m = c.abs() / unit
        best = torch.zeros_like(m, dtype=torch.int64)
        dist = m.clone()
        for n in range(1, 8):
            far = (m - grid[n]).abs()
            nearer = (far < dist) | ((far == dist) & (n % 2 == 0))
            best = torch.where(nearer, n, best)
            dist = torch.where(nearer, far, dist)
        out[at:at + (1 << 20)] = torch.copysign(grid[best], c) * unit
    return out.view(*v.shape[:-1], K)


def _decoded(raw, N, K):
    """One matrix's values in 64 bits, from its bytes."""
    table = torch.tensor(_TABLE, dtype=torch.float64, device=raw.device)
    codes = raw[:N * K // 2].view(N, K // 2).int()
    w = torch.empty(N, K, dtype=torch.float64, device=raw.device)
    w[:, 0::2] = table[codes & 15]
    w[:, 1::2] = table[codes >> 4]
    r = torch.arange(N, device=raw.device)[:, None]
    b = torch.arange(K // 32, device=raw.device)[None, :]
    at = (r // 128 * (K // 128) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    return w * torch.exp2(raw[N * K // 2:][at].double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        l = torch.cat([torch.einsum("ed,td->te", s["w"].double(), s["x"][t:t + 2048].double()) for t in range(0, T, 2048)])
        if case["scoring"] == "sigmoid":
            score = 1 / (1 + torch.exp(-l))
        else:
            p = torch.exp(l - l.max(1, keepdim=True)[0])
            score = p / p.sum(1, keepdim=True)
        c = score.clone() if s["bias"] is None else score + s["bias"].double()
        low = torch.full((T, 1), -math.inf, dtype=torch.float64, device=c.device)
        if G > 1:
            left, total = c.reshape(T, G, E // G).clone(), 0
            for _ in range(case["group_top"]):
                v, i = left.max(2, keepdim=True)
                total = total + v[..., 0]
                left.scatter_(2, i, -math.inf)
            out = torch.ones(T, G, dtype=torch.bool, device=c.device)
            for _ in range(case["kept"]):
                g = total.argmax(1, keepdim=True)
                out.scatter_(1, g, False)
                total.scatter_(1, g, low)
            c = c.masked_fill(out.repeat_interleave(E // G, 1), -math.inf)
        picks = []
        for _ in range(k):
            e = c.argmax(1, keepdim=True)
            picks.append(e)
            c.scatter_(1, e, low)
        idx = torch.cat(picks, 1)
        w = score.gather(1, idx)
        return {"idx": idx.int(), "w": w * (case["scale"] / w.sum(1, keepdim=True) if case["renorm"] else case["scale"])}
    if op == "quantize":
        v = _nearest(s["x"].double())
        return v if s["perm"] is None else v[s["perm"].long() // case["k"]]
    bounds = s["offsets"].tolist()
    if op == "product":
        N, K = case["N"], case["K"]
        table = torch.tensor(_TABLE, dtype=torch.float64, device="cuda")
        x = torch.stack([table[(s["codes"] & 15).int()], table[(s["codes"] >> 4).int()]], -1).view(-1, K // 32, 32)
        x = (x * torch.exp2(s["scales"].double() - 127)[..., None]).view(-1, K)
        y = torch.empty(x.shape[0], N, dtype=torch.float64, device="cuda")
        for e in s["active"].tolist():
            y[bounds[e]:bounds[e + 1]] = x[bounds[e]:bounds[e + 1]] @ _decoded(s["mats"][e], N, K).t()
        return y
    d, F = case["d"], case["F"]
    x = _nearest(s["x"].double())[s["perm"].long() // case["k"]]
    y = torch.empty(x.shape[0], d, dtype=torch.float64, device="cuda")
    split = F * d + F * d // 16
    for e in s["active"].tolist():
        gu = _decoded(s["blobs"][e, :split], 2 * F, d)
        rows = torch.arange(2 * F, device="cuda")
        xe = x[bounds[e]:bounds[e + 1]]
        gate, up = xe @ gu[rows % 64 < 32].t(), xe @ gu[rows % 64 >= 32].t()
        h = _nearest(gate / (1 + torch.exp(-gate)) * up)
        y[bounds[e]:bounds[e + 1]] = h @ _decoded(s["blobs"][e, split:], d, F).t()
    return y
