"""GPU parity of the router (top-k, weights, row plan) and of the row sort, against the plain 64-bit form: choices and
plans equal, ties to the lowest expert, masked experts and rows that are masked whole, weights within fp32 rounding."""
import numpy as np
import pytest
import torch

import opref
import w4a4_mxfp4_quantized_b200 as mq
from sfutil import Guarded

pytestmark = pytest.mark.gpu


def check(logits, topk, sigmoid=False, renorm=True, scale=1.0):
    T, E = logits.shape
    o = [Guarded(T * topk * 4, dtype=torch.float32, shape=(T, topk)), Guarded(T * topk * 4, dtype=torch.int32, shape=(T, topk)),
         Guarded((E + 1) * 4, dtype=torch.int32), Guarded(T * topk * 4, dtype=torch.int32),
         Guarded(T * topk * 4, dtype=torch.int32, shape=(T, topk))]
    got = mq.moe_route(logits, topk, scoring=mq.SCORE_SIGMOID if sigmoid else mq.SCORE_SOFTMAX, renormalize=renorm, scale=scale,
                       weights=o[0].t, ids=o[1].t, group_offsets=o[2].t, row_index=o[3].t, pos=o[4].t)
    torch.cuda.synchronize()
    assert all(g.intact() for g in o), "write outside an output"
    w, tol, ids = opref.route(logits.double().cpu().numpy(), topk, sigmoid, renorm, scale)
    np.testing.assert_array_equal(got[1].cpu().numpy(), ids)
    off, row, pos = opref.groups(ids.tolist(), E)
    np.testing.assert_array_equal(got[2].cpu().numpy(), off)
    np.testing.assert_array_equal(got[3].cpu().numpy(), row)
    np.testing.assert_array_equal(got[4].cpu().numpy(), pos)
    err = np.abs(got[0].cpu().double().numpy() - w)
    assert np.all(err <= tol * np.abs(w) + 2.0 ** -140), float(np.max(err / (np.abs(w) + 1e-300)))


def logits_of(seed, T, E, dtype=torch.float32, spread=2.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * spread).to(dtype)


@pytest.mark.parametrize("T,E,topk", [(1, 128, 8), (3, 1, 1), (64, 128, 8), (257, 72, 6), (700, 257, 5), (33, 1024, 32),
                                      (2500, 33, 3), (31, 32, 32), (300, 512, 9)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sizes(T, E, topk, dtype):
    check(logits_of(T + E, T, E, dtype), topk)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_scorings(sigmoid, renorm):
    check(logits_of(5, 129, 96, spread=6.0), 7, sigmoid, renorm, scale=2.5)


def test_ties_go_to_the_lowest_expert():
    g = torch.Generator("cuda").manual_seed(1)
    l = torch.randint(-2, 3, (200, 100), generator=g, device="cuda").float()
    l[::7] = 0.25
    l[3, ::2] = -0.0
    l[3, 1::2] = 0.0
    check(l, 10)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_experts_rows_and_odd_values(sigmoid, renorm):
    l = logits_of(9, 60, 40)
    l[:, 5:30] = -float("inf")
    l[10] = -float("inf")            # nothing left
    l[11] = float("nan")
    l[12, 1:] = -float("inf")        # one expert left
    l[13, 3] = float("nan")
    l[14, :2] = float("inf")         # two largest
    l[15] = -3.0e38
    l[16] = torch.linspace(-200.0, -100.0, 40, device="cuda")   # every sigmoid underflows
    l[17] = torch.finfo(torch.float32).min                       # the type's lowest value is not a mask
    check(l, 6, sigmoid, renorm)


def test_strided_rows_and_no_rows():
    wide = logits_of(3, 50, 200, torch.bfloat16)
    check(wide[:, 17:17 + 90], 4)
    w, ids, off, row, pos = mq.moe_route(torch.empty(0, 64, device="cuda"), 4)
    torch.cuda.synchronize()
    assert w.shape == (0, 4) and row.numel() == 0 and bool((off == 0).all())


def check_groups(ids, E):
    R = ids.numel()
    o = [Guarded((E + 1) * 4, dtype=torch.int32), Guarded(R * 4, dtype=torch.int32), Guarded(R * 4, dtype=torch.int32, shape=ids.shape)]
    off, row, pos = mq.row_groups(ids, E, group_offsets=o[0].t, row_index=o[1].t, pos=o[2].t)
    torch.cuda.synchronize()
    assert all(g.intact() for g in o)
    want = opref.groups(ids.reshape(ids.shape[0], -1).tolist(), E)
    np.testing.assert_array_equal(off.cpu().numpy(), want[0])
    np.testing.assert_array_equal(row.cpu().numpy(), want[1])
    np.testing.assert_array_equal(pos.cpu().numpy().reshape(want[2].shape), want[2])


@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (64, 1, 32), (31, 3, 5), (1024, 8, 128), (8747, 8, 1024), (40000, 1, 3), (65, 1, 1024),
                                      (1, 1500, 7)])
def test_row_groups(T, topk, E):
    g = torch.Generator("cuda").manual_seed(T + E)
    ids = torch.randint(-2, E + 2, (T, topk), generator=g, device="cuda", dtype=torch.int32)   # repeats, and ids of no group
    check_groups(ids, E)


def test_row_groups_edges():
    check_groups(torch.full((300,), -1, dtype=torch.int32, device="cuda"), 4)            # nothing in a group
    check_groups(torch.full((300,), 3, dtype=torch.int32, device="cuda"), 4)             # everything in the last
    off, row, pos = mq.row_groups(torch.empty(0, dtype=torch.int32, device="cuda"), 9)
    torch.cuda.synchronize()
    assert bool((off == 0).all()) and off.numel() == 10
    ids = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1], dtype=torch.int32, device="cuda")
    check_groups(ids, 2)


def test_captured_and_replayed_with_new_logits():
    l = logits_of(1, 300, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mq.moe_route(l, 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mq.moe_route(l, 4)
    for seed in (2, 3):
        l.copy_(logits_of(seed, 300, 64))
        graph.replay()
        torch.cuda.synchronize()
        want = mq.moe_route(l.clone(), 4)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_the_plan_feeds_the_grouped_calls():
    """Dispatch and combine through moe_route's plan equal the token-order computation: an identity expert."""
    T, E, topk, K = 200, 16, 3, 256
    X = torch.randn(T, K, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).to(torch.bfloat16)
    l = logits_of(8, T, E)
    l[50:60] = -float("inf")
    w, ids, off, row, pos = mq.moe_route(l, topk)
    live = int(off[-1])
    assert live == (T - 10) * topk
    out = mq.moe_combine(X[row.long()][:live].contiguous(), pos, w, out_dtype=mq.OUT_F32)
    q, sf = mq.act_quant_gather(X, row, None, 32, group_offsets=off)
    want_q, _ = mq.act_quant(X[row.long()].contiguous(), None, 32, group_offsets=off)
    torch.cuda.synchronize()
    assert torch.equal(q[:live], want_q[:live])
    ref = X.double() * w.double().sum(1, keepdim=True)
    assert bool(((out.double() - ref).abs() <= (2 * topk + 1) * opref.F32 * X.double().abs()).all())
    assert bool((out[50:60] == 0).all())
