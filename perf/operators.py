"""Measured cases of the MXFP4-activation operators and of the verification
step from probabilities.

Four operators, each in a plain form (elementary torch operations in fp32, fp64
where a decision hangs on a long sum) and, where `own` is true, as the call a
user makes of the library:

  gemm       C[m, n] = sum_k A[m, k] B[n, k], both factors MXFP4
  gate_up    h_r = silu(W_gate x_t) * (W_up x_t) for the rows r of every expert,
             x and W MXFP4, t = sorted_pairs[r] / k
  down       y_r = W_down h_r for the rows r of every expert, h and W MXFP4
  verify     acceptance of drafted tokens and the draw of the next one from
             probabilities

Sizes are those of the page-shaped layer (hidden 6144, 384 experts, 8 active,
intermediate 2048, vocabulary 152064, blocks of 8) and odd ones."""

import math

import torch

own = False

H, I, E, K8, V = 6144, 2048, 384, 8, 152064
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one drafted block of 8 tokens through a dense projection: latency
        {"name": "gemm_t8", "op": "gemm", "M": 8, "N": 4096, "K": 6144, "out": "bf16"},
        # a ragged batch: rows, columns and the last K step all partial
        {"name": "gemm_odd", "op": "gemm", "M": 333, "N": 1001, "K": 2080, "out": "f32"},
        # 64 blocks of 8 through an expert-sized output projection
        {"name": "gemm_t512", "op": "gemm", "M": 512, "N": 6144, "K": 2048, "out": "bf16"},
        # a prefill chunk through a gate/up-sized projection: matrix-core bound
        {"name": "gemm_t8192", "op": "gemm", "M": 8192, "N": 4096, "K": 6144, "out": "f32"},
        # one verify step: nearly every chosen expert has one row
        {"name": "gate_up_t8", "op": "gate_up", "T": 8, "H": H, "I": I, "E": E, "k": K8, "zipf": 0.0},
        # 64 sequences with skewed expert popularity: one-row and hundred-row experts together
        {"name": "gate_up_zipf_t512", "op": "gate_up", "T": 512, "H": H, "I": I, "E": E, "k": K8, "zipf": 1.1},
        # a prefill chunk: about 170 rows an expert
        {"name": "gate_up_t8192", "op": "gate_up", "T": 8192, "H": H, "I": I, "E": E, "k": K8, "zipf": 0.0},
        # a verify step of 8 sequences
        {"name": "down_t64", "op": "down", "T": 64, "H": H, "I": I, "E": E, "k": K8, "zipf": 0.0},
        # a small layer with sizes that are multiples of 32 and of nothing more
        {"name": "down_odd", "op": "down", "T": 257, "H": 1056, "I": 352, "E": 24, "k": 3, "zipf": 0.6},
        # a prefill chunk
        {"name": "down_t8192", "op": "down", "T": 8192, "H": H, "I": I, "E": E, "k": K8, "zipf": 0.0},
        # one drafted block, plain softmax probabilities: latency
        {"name": "verify_one", "op": "verify", "B": 1, "L": 8, "V": V, "type": "f32", "ragged": False, "filtered": False},
        # 64 sequences with blocks of unequal length and truncated (min-p) target probabilities
        {"name": "verify_b64", "op": "verify", "B": 64, "L": 8, "V": V, "type": "bf16", "ragged": True, "filtered": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gate_up", "down", "verify"])
    if op == "gemm":
        return {"op": op, "M": _log_int(rng, 1, 8192), "N": _log_int(rng, 1, 6144),
                "K": 32 * _log_int(rng, 1, 128), "out": rng.choice(["f32", "bf16"])}
    if op == "verify":
        return {"op": op, "B": _log_int(rng, 1, 64), "L": rng.randint(1, 12), "V": _log_int(rng, 16, V),
                "type": rng.choice(["f32", "bf16"]), "ragged": rng.random() < 0.5, "filtered": rng.random() < 0.5}
    experts = _log_int(rng, 1, E)
    return {"op": op, "T": _log_int(rng, 1, 8192), "H": 32 * _log_int(rng, 1, H // 32), "I": 32 * _log_int(rng, 1, I // 32),
            "E": experts, "k": rng.randint(1, min(8, experts)), "zipf": rng.choice([0.0, 0.6, 1.1])}


# ---- inputs ------------------------------------------------------------------

def _quantise(x):
    """x [rows, K] f32 -> MXFP4 (codes [rows, K/2], scales [rows, K/32]): OCP MX v1.0, ties to the even code."""
    rows, k = x.shape
    b = x.view(rows, k // 32, 32)
    amax = b.abs().amax(2)
    e = (torch.frexp(amax).exponent - 1 - 2 + 127).clamp(0, 254)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    m = torch.ldexp(b, (127 - e).unsqueeze(2)).abs()
    c = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    c = (c + 8 * (b < 0).to(torch.uint8)).view(rows, k // 2, 2)
    return (c[..., 0] + 16 * c[..., 1]).to(torch.uint8), e.to(torch.uint8)


def _weights(shape, k, g):
    """Uniform E2M1 codes and block exponents 2^-9 .. 2^-3, as the page-shaped layer's weights are drawn."""
    codes = torch.randint(0, 256, (*shape, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(118, 125, (*shape, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales


def _routing(case, g):
    """Expert lists of a batch: rows sorted by expert, ascending pair ids within one."""
    t, e, k = case["T"], case["E"], case["k"]
    logits = 1.5 * torch.randn(t, e, device="cuda", generator=g)
    if case["zipf"]:
        rank = torch.randperm(e, device="cuda", generator=g) + 1
        logits = logits - case["zipf"] * rank.float().log()
    ids = logits.topk(k, dim=1).indices.view(-1)
    order = torch.sort(ids, stable=True).indices
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.bincount(ids, minlength=e).cumsum(0)
    return order.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "gemm":
        m, n, k = case["M"], case["N"], case["K"]
        s["a"] = _quantise(torch.randn(m, k, device="cuda", generator=g))
        s["b"] = _weights((n,), k, g)
        s["out"] = torch.empty(m, n, dtype=DTYPES[case["out"]], device="cuda")
    elif case["op"] == "gate_up":
        s["x"] = _quantise(torch.randn(case["T"], case["H"], device="cuda", generator=g))
        s["pairs"], s["offsets"] = _routing(case, g)
        s["k"] = case["k"]
        s["w"] = _weights((case["E"], 2 * case["I"]), case["H"], g)
        s["out"] = torch.empty(case["T"] * case["k"], case["I"], dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "down":
        r = case["T"] * case["k"]
        u = torch.randn(r, case["I"], device="cuda", generator=g)
        s["h"] = _quantise(u * torch.randn(r, case["I"], device="cuda", generator=g).abs())
        s["pairs"], s["offsets"] = _routing(case, g)
        s["k"] = case["k"]
        s["w"] = _weights((case["E"], case["H"]), case["I"], g)
        s["out"] = torch.empty(r, case["H"], dtype=torch.float32, device="cuda")
    else:
        b, l, v = case["B"], case["L"], case["V"]
        logits = 3.0 * torch.randn(b, l + 1, v, device="cuda", generator=g)
        q = torch.softmax(logits[:, :l] + 0.35 * torch.randn(b, l, v, device="cuda", generator=g), 2)
        p = torch.softmax(logits, 2)
        if case["filtered"]:
            p = torch.where(p >= 0.02 * p.amax(2, keepdim=True), p, torch.zeros_like(p))
            p = p / p.sum(2, keepdim=True)
        s["tokens"] = torch.multinomial(q.view(b * l, v), 1, generator=g).view(b, l).to(torch.int32)
        s["p"], s["q"] = p.to(DTYPES[case["type"]]), q.to(DTYPES[case["type"]])
        s["u"] = torch.rand(b, l + 1, device="cuda", generator=g)
        s["len"] = torch.randint(0, l + 1, (b,), dtype=torch.int32, device="cuda", generator=g) if case["ragged"] else None
        s["out"] = [torch.empty(b, dtype=torch.int32, device="cuda") for _ in range(2)]
    return s


# ---- one pass ------------------------------------------------------------------

def _dequant(codes, scales):
    """MXFP4 -> fp32, exact."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    lut = torch.cat([lut, -lut])
    pair = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)          # both nibbles of a byte
    v = pair[codes.int()].view(*codes.shape[:-1], -1, 32)
    return (v * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).flatten(-2)


def _plain_experts(s, f, rows):
    off = s["offsets"].tolist()
    codes, scales = s["w"]
    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            s["out"][lo:hi] = f(rows(lo, hi) @ _dequant(codes[e], scales[e]).t())
    return s["out"]


def _swiglu(gu):
    i = gu.shape[1] // 2
    g, u = gu[:, :i], gu[:, i:]
    return (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)


def _clean(v):
    """Probabilities in fp64; what is not a positive finite number counts as none."""
    v = v.double()
    return torch.where((v > 0) & (v < math.inf), v, torch.zeros_like(v))


def _plain_verify(s):
    p, q, d, u = s["p"], s["q"], s["tokens"].long(), s["u"].double()
    b, l, v = q.shape
    n_max = torch.full((b,), l, device=p.device) if s["len"] is None else s["len"].long().clamp(0, l)
    at = d.clamp(0, v - 1).unsqueeze(2)
    pd, qd = _clean(p[:, :l].gather(2, at))[..., 0], _clean(q.gather(2, at))[..., 0]
    ok = (d >= 0) & (d < v) & (u[:, :l] * qd < pd) & (torch.arange(l, device=p.device) < n_max.unsqueeze(1))
    n = ok.int().cumprod(1).sum(1)
    seq = torch.arange(b, device=p.device)
    pn = _clean(p[seq, n])
    w = (pn - _clean(q[seq, n.clamp(max=l - 1)])).clamp(min=0)
    w = torch.where(((n < n_max) & (w.amax(1) > 0)).unsqueeze(1), w, pn)
    c = w.cumsum(1)
    token = (c <= u[:, l:] * c[:, -1:]).sum(1)
    return [n.int(), torch.where(c[:, -1] > 0, token, torch.full_like(token, -1)).int()]


def run(s):
    if own:
        import mxfp4_moe_expert_route_amd as mm
        if s["op"] == "gemm":
            return mm.mxfp4_gemm(*s["a"], *s["b"], dtype=s["out"].dtype, out=s["out"])
        if s["op"] == "gate_up":
            return mm.moe_mxfp4_a4_gate_up_swiglu(*s["x"], s["pairs"], s["offsets"], s["k"], *s["w"], h=s["out"])
        if s["op"] == "down":
            return mm.moe_mxfp4_a4_down(*s["h"], s["offsets"], s["k"], *s["w"], y=s["out"])
        return mm.dflash_verify_probs(s["p"], s["q"], s["tokens"], s["u"], draft_len=s["len"],
                                      accept_len=s["out"][0], next_token=s["out"][1])
    if s["op"] == "gemm":
        return (_dequant(*s["a"]) @ _dequant(*s["b"]).t()).to(s["out"].dtype)
    if s["op"] == "gate_up":
        x = _dequant(*s["x"])
        return _plain_experts(s, _swiglu, lambda lo, hi: x[(s["pairs"][lo:hi] // s["k"]).long()])
    if s["op"] == "down":
        h = _dequant(*s["h"])
        return _plain_experts(s, lambda y: y, lambda lo, hi: h[lo:hi])
    return _plain_verify(s)


# ---- what a pass cannot do without ------------------------------------------------

def _touched(case):
    """Expected number of experts with rows."""
    e, pairs = case["E"], case["T"] * case["k"]
    p = [(r + 1.0) ** -case["zipf"] for r in range(e)]
    total = sum(p)
    return min(e, pairs, sum(1.0 - (1.0 - x / total) ** pairs if e > 1 else 1.0 for x in p))


def work(case):
    row = lambda k: k / 2 + k / 32  # noqa: E731  bytes of an MXFP4 row
    if case["op"] == "gemm":
        m, n, k = case["M"], case["N"], case["K"]
        return {"bytes": (m + n) * row(k) + m * n * (4 if case["out"] == "f32" else 2), "flops": 2.0 * m * n * k}
    if case["op"] == "verify":
        size = 4 if case["type"] == "f32" else 2      # one row of p and of q, the drafted tokens' entries
        return {"bytes": case["B"] * (2.0 * case["V"] * size + case["L"] * (8 + 2 * size) + 16), "flops": 4.0 * case["B"] * case["V"]}
    r, h, i, w = case["T"] * case["k"], case["H"], case["I"], _touched(case)
    if case["op"] == "gate_up":
        return {"bytes": w * 2 * i * row(h) + case["T"] * row(h) + 4 * r + 2 * r * i, "flops": 4.0 * r * h * i}
    return {"bytes": w * h * row(i) + r * row(i) + 4 * r * h, "flops": 2.0 * r * h * i}


# ---- the definition, in 64 bits ----------------------------------------------------

def _values(codes, scales):
    """Element values from the bit fields: sign, two exponent bits of bias 1, one mantissa bit; block factor 2^(e-127)."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    man, ex = (n & 1).double(), ((n >> 1) & 3).double()
    mag = torch.where(ex > 0, (1.0 + 0.5 * man) * 2.0 ** (ex - 1.0), 0.5 * man)
    block = (2.0 ** (scales.double() - 127.0)).repeat_interleave(32, -1)
    return torch.where(n >= 8, -mag, mag) * block


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        return _values(*s["a"]) @ _values(*s["b"]).t()
    if case["op"] == "verify":
        return _exact_verify(s)
    src = _values(*(s["x"] if case["op"] == "gate_up" else s["h"]))
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    bounds = s["offsets"].cpu().numpy()
    for e in range(case["E"]):
        rows = torch.arange(bounds[e], bounds[e + 1], device="cuda")
        if not len(rows):
            continue
        w = _values(s["w"][0][e], s["w"][1][e])
        if case["op"] == "down":
            out[rows] = src[rows] @ w.t()
        else:
            x = src[torch.div(s["pairs"][rows].long(), case["k"], rounding_mode="floor")]
            out[rows] = torch.nn.functional.silu(x @ w[:case["I"]].t()) * (x @ w[case["I"]:].t())
    return out


def _exact_verify(s):
    l = s["q"].shape[1]
    accepted, token = [], []
    for b in range(s["p"].shape[0]):
        p, q, u = s["p"][b].double(), s["q"][b].double(), s["u"][b].tolist()
        most = l if s["len"] is None else int(s["len"][b])
        n = 0
        for d in s["tokens"][b].tolist()[:most]:
            if not u[n] * float(q[n, d]) < float(p[n, d]):
                break
            n += 1
        w = torch.relu(p[n] - q[n]) if n < most else p[n]
        w = w if float(w.sum()) > 0 else p[n]
        c = torch.cumsum(w, 0)
        accepted.append(n)
        token.append(int(torch.searchsorted(c, u[l] * c[-1], right=True)))
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (accepted, token)]
