"""The layer routed by scores at thousands of tokens: its separate calls bit for bit
(k = 8, whose grouping starts from the routing's counts, and others), and the oracle's
experts mixed by the oracle's routing on a sample of tokens."""

import numpy as np
import pytest
import torch

import workloads
from _gpu import DEV, dev_bf16, dev_u8, say, tol_check
from oracle import layer as olayer
from oracle import scored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    import mxfp4_moe_expert_route_amd as m
    m._lib.lib()
    return m


@pytest.mark.parametrize("T,k,sigmoid", [(4100, 8, True), (8192, 8, False), (5001, 3, True), (4096, 6, False)])
def test_layer(mm, T, k, sigmoid):
    say("scored layer, many tokens", T, k, sigmoid)
    E = 24
    c = workloads.custom_config("scored", 92, T, 256, 128, E, k)
    w = workloads.all_weights(c, 0)
    dev = [dev_u8(w[n]) for n in ("w13_codes", "w13_scales", "w2_codes", "w2_scales")]
    rng = np.random.default_rng([T, k])
    xb = workloads.gen_x_bits(c, 0)
    logits, bias = rng.normal(0, 1, (T, E)).astype(np.float32), (rng.integers(-60, 61, E) / 8192).astype(np.float32)
    logits[::97, 2:] = -np.inf                            # two experts left
    logits[5::101] = np.nan                               # none
    rule = dict(score="sigmoid" if sigmoid else "softmax", groups=4, topk_groups=2, group_best=2, scale=2.5)
    x, lg, bt = dev_bf16(xb), torch.from_numpy(logits).to(DEV), torch.from_numpy(bias).to(DEV)
    b = mm.LayerBuffers(T, c.H, c.I, E, k, DEV)
    for v in (b.h, b.y, b.out):
        v.fill_(7.0)
    b.workspace.fill_(0xff)
    mm.moe_mxfp4_scored_layer(x, lg, k, *dev, bias=bt, **rule, buffers=b)
    ids, wt = mm.moe_route_scored(lg, k, bias=bt, **rule)
    counts, offsets, pairs, row = mm.moe_permute(ids, E)
    n = int(offsets[-1])
    assert n < k * T
    h, y = torch.full_like(b.h, 7.0), torch.full_like(b.y, 7.0)
    mm.moe_mxfp4_gate_up_swiglu(x, pairs, offsets, k, dev[0], dev[1], h=h)
    mm.moe_mxfp4_down(h, offsets, k, dev[2], dev[3], y=y)
    out = mm.moe_combine(y, wt, row)
    for a, e in ((b.topk_ids, ids), (b.topk_w, wt), (b.counts, counts), (b.offsets, offsets), (b.pair_to_row, row),
                 (b.sorted_pairs[:n], pairs[:n]), (b.h, h), (b.y, y), (b.out, out)):
        assert torch.equal(a, e)
    assert (b.y[n:] == 7.0).all() and (b.h[n:] == 7.0).all()
    assert not b.out[5::101].any()
    some = np.concatenate([[0, 97, 5, 106, T - 1], rng.permutation(T)[:35]])
    oid, ow = scored.route(logits[some], k, bias, sigmoid, groups=4, keep=2, scale=2.5)
    assert np.array_equal(ids.cpu().numpy()[some], oid)
    full = olayer.layer_forward(xb[some], np.tile(-np.arange(E, dtype=np.float32), (len(some), 1)), w["w13_codes"],
                                w["w13_scales"], w["w2_codes"], w["w2_scales"], E)
    each = np.asarray(full["y"], np.float64).reshape(len(some), E, c.H)    # slot j holds expert j
    want = sum(ow[:, j, None] * each[np.arange(len(some)), np.maximum(oid[:, j], 0)] for j in range(k))
    tol_check(b.out.cpu().numpy()[some], want, "scored layer out")
