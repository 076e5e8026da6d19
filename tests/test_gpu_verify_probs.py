"""GPU parity of dflash_verify_probs with the float64 oracle.

Acceptance is exact on both sides.  Sums are float64 on both sides, in
different orders, so a draw could differ only within 2^-35 of a boundary,
which no input here comes near: results are required to be equal."""

import numpy as np
import pytest
import torch

from _gpu import DEV, say
from oracle import mx as omx
from oracle import verify_probs as ovp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


def inputs(rng, B, L, V, filtered):
    logits = rng.normal(0, 3, (B, L + 1, V))
    soft = lambda z: np.exp(z - z.max(2, keepdims=True)) / np.exp(z - z.max(2, keepdims=True)).sum(2, keepdims=True)  # noqa: E731
    p, q = soft(logits), soft(logits[:, :L] + rng.normal(0, 0.35, (B, L, V)))
    if filtered:
        p = np.where(p >= 0.02 * p.max(2, keepdims=True), p, 0.0)
        p /= p.sum(2, keepdims=True)
    c = np.cumsum(q, 2)
    tokens = np.minimum((c <= rng.random((B, L, 1)) * c[:, :, -1:]).sum(2), V - 1).astype(np.int32)
    u = np.minimum(rng.random((B, L + 1)), 1.0 - 2.0 ** -24).astype(np.float32)
    return p, q, tokens, u


def store(v, dtype):
    """(device tensor, the float64 values it holds)"""
    if dtype == torch.float32:
        v = v.astype(np.float32)
        return torch.from_numpy(v).to(DEV), v.astype(np.float64)
    bits = omx.to_bf16_bits(v)
    t = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).to(DEV)
    return t, omx.bf16_bits_to_f64(bits)


def check(mm, p, q, tokens, u, lengths, dtype):
    pt, p64 = store(p, dtype)
    qt, q64 = store(q, dtype)
    n, t = ovp.verify(p64, q64, tokens, u, lengths)
    dl = None if lengths is None else torch.from_numpy(np.asarray(lengths, np.int32)).to(DEV)
    gn, gt = mm.dflash_verify_probs(pt, qt, torch.from_numpy(tokens).to(DEV), torch.from_numpy(u).to(DEV), draft_len=dl)
    assert np.array_equal(gn.cpu().numpy(), n)
    assert np.array_equal(gt.cpu().numpy(), t)
    return n, t


SIZES = [(1, 1, 1), (3, 2, 2), (5, 1, 3), (7, 8, 64), (4, 32, 100), (2, 8, 1000), (70, 3, 257), (6, 8, 1024),
         (3, 8, 5001), (9, 5, 20011), (600, 2, 300), (2, 8, 152064), (1, 2, 16385), (130, 1, 17001), (1, 1, 65536),
         (513, 1, 17000),
         (4, 3, 2048), (4, 3, 2049), (5, 2, 8192), (5, 2, 8193), (520, 1, 8200)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,L,V", SIZES)
def test_matches_oracle(mm, B, L, V, dtype):
    say("verify_probs", B, L, V, dtype)
    for seed, filtered in ((0, False), (1, True)):
        rng = np.random.default_rng([B, L, V, seed])
        p, q, tokens, u = inputs(rng, B, L, V, filtered)
        lengths = rng.integers(-1, L + 2, B) if filtered else None      # clamped to 0..L
        check(mm, p, q, tokens, u, lengths, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 300, 2049, 4099, 8300, 20000])
def test_edges(mm, V, dtype):
    say("verify_probs edges", V, dtype)
    rng = np.random.default_rng(V)
    B, L = 12, 4
    p, q, tokens, u = inputs(rng, B, L, V, False)
    q[0], tokens[0] = p[0, :L], p[0, :L].argmax(1)           # equal distributions: all accepted
    u[0, :L] = 1.0 - 2.0 ** -24
    q[1], tokens[1, 0] = p[1, :L], -1                        # no residual, token rejected: drawn from p
    tokens[2, 1], tokens[3, 0] = V, 2 ** 30                  # outside the vocabulary
    p[4, 0] = 0.0                                            # nothing to draw from
    p[5, 0], q[5, 0] = 0.0, 0.0
    p[5, 0, V - 1] = 1.0                                     # one-hot at the end
    p[6, 0, :3] = [np.nan, -0.5, np.inf]                     # count as none
    q[6, 0, :3] = [np.inf, np.nan, -1.0]
    tokens[6, 0] = 2
    u[7, L], u[8, L] = 0.0, 1.0 - 2.0 ** -24                 # the first and the last token with weight
    tokens[7, 0] = tokens[8, 0] = -5
    p[8, 0, V // 2:] = 0.0
    p[9] *= 1e-30                                            # far from normalised
    q[9] *= 1e-30
    p[10] = 0.0
    p[10, :, V // 3] = 2.0 ** -126
    tokens[10] = V // 3
    u[11] = 0.0
    lengths = np.full(B, L)
    lengths[11] = 0
    n, t = check(mm, p, q, tokens, u, lengths, dtype)
    assert n[0] == L and n[1] == 0 and n[4] == 0 and t[4] == -1 and t[5] == V - 1 and n[11] == 0


def test_outputs_workspace_and_refusals(mm):
    say("verify_probs buffers and refusals")
    rng = np.random.default_rng(2)
    B, L, V = 6, 3, 20000
    p, q, tokens, u = inputs(rng, B, L, V, False)
    args = [torch.from_numpy(p.astype(np.float32)).to(DEV), torch.from_numpy(q.astype(np.float32)).to(DEV),
            torch.from_numpy(tokens).to(DEV), torch.from_numpy(u).to(DEV)]
    n, t = mm.dflash_verify_probs(*args)
    ws = torch.full((mm.dflash_verify_probs_workspace_bytes(B, L, V),), 0xff, dtype=torch.uint8, device=DEV)
    a, b = (torch.full((B,), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    mm.dflash_verify_probs(*args, accept_len=a, next_token=b, workspace=ws)     # garbage in the workspace
    assert torch.equal(a, n) and torch.equal(b, t)
    with pytest.raises(mm._lib.MxmError):
        mm.dflash_verify_probs(*args, workspace=ws[:8])
    with pytest.raises(TypeError):
        mm.dflash_verify_probs(args[0].bfloat16(), *args[1:])
    with pytest.raises(ValueError):
        mm.dflash_verify_probs(args[0][:, :L].contiguous(), *args[1:])
    with pytest.raises(ValueError):
        mm.dflash_verify_probs(*args, draft_len=torch.zeros(B + 1, dtype=torch.int32, device=DEV))
    empty = mm.dflash_verify_probs(*[v[:0] for v in args])
    assert empty[0].numel() == 0 and empty[1].numel() == 0


def test_captured_and_replayed(mm):
    say("verify_probs replays")
    rng = np.random.default_rng(4)
    B, L, V = 5, 8, 20000
    sets = []
    for _ in range(2):
        p, q, tokens, u = inputs(rng, B, L, V, True)
        s = [torch.from_numpy(p.astype(np.float32)).to(DEV), torch.from_numpy(q.astype(np.float32)).to(DEV),
             torch.from_numpy(tokens).to(DEV), torch.from_numpy(u).to(DEV)]
        sets.append((s, [v.clone() for v in mm.dflash_verify_probs(*s)]))
    live = [v.clone() for v in sets[0][0]]
    ws = torch.zeros(mm.dflash_verify_probs_workspace_bytes(B, L, V), dtype=torch.uint8, device=DEV)
    out = [torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mm.dflash_verify_probs(*live, accept_len=out[0], next_token=out[1], workspace=ws)
    for i in range(4):
        for dst, src in zip(live, sets[i % 2][0]):
            dst.copy_(src)
        out[0].zero_()
        out[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], sets[i % 2][1][0]) and torch.equal(out[1], sets[i % 2][1][1]), i


@pytest.mark.parametrize("V", [3, 2500])
def test_largest_batch(mm, V):
    """2^20 blocks, both one-launch forms.  Probabilities are multiples of 1/4
    and uniforms of 2^-10, so every sum and comparison is exact."""
    say("verify_probs, 2^20 blocks", V)
    B = 1 << 20
    g = torch.Generator(device=DEV).manual_seed(V)
    p, q = (torch.randint(0, 5, (B, n, V), device=DEV, generator=g, dtype=torch.int8).to(torch.bfloat16) / 4
            for n in (2, 1))
    tokens = torch.randint(0, V, (B, 1), device=DEV, generator=g).int()
    u = torch.randint(0, 1024, (B, 2), device=DEV, generator=g).float() / 1024
    n, t = mm.dflash_verify_probs(p, q, tokens, u)
    for b0 in range(0, B, 1 << 16):
        rows = slice(b0, min(b0 + (1 << 16 if V < 100 else 2048), B))      # of the larger, part
        pr, qr, d = p[rows].float(), q[rows, 0].float(), tokens[rows].long()
        accept = u[rows, :1] * qr.gather(1, d) < pr[:, 0].gather(1, d)
        rest = (pr[:, 0] - qr).clamp_min(0)
        rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, pr[:, 0])
        w = torch.where(accept, pr[:, 1], rest)
        cum = w.cumsum(1)
        total = cum[:, -1:]
        want = torch.where(total > 0, (cum <= u[rows, 1:] * total).sum(1, keepdim=True), -1)
        assert torch.equal(n[rows], accept[:, 0].int())
        assert torch.equal(t[rows], want[:, 0].int())
