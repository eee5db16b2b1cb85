"""GPU parity of the few-token expert layer (gate/up, SwiGLU, down, weighted combine on MXFP4 weights) against the plain
64-bit form, within its carried rounding bound; ragged routing, dropped choices, every Hadamard block, extreme scales."""
import numpy as np
import pytest
import torch

import opref
import w4a4_mxfp4_quantized_b200 as mq
from sfutil import Guarded, swizzle

pytestmark = pytest.mark.gpu


def layer_of(seed, E, K, I, N, b=32, b_dn=32, scaled=True, lo=115, hi=119):
    rng = np.random.default_rng(seed)
    d = dict(wq_gu=rng.integers(0, 256, (E, 2 * I, K // 2), dtype=np.uint8), sf_gu=rng.integers(lo, hi, (E, 2 * I, K // 32), dtype=np.uint8),
             wq_dn=rng.integers(0, 256, (E, N, I // 2), dtype=np.uint8), sf_dn=rng.integers(lo, hi, (E, N, I // 32), dtype=np.uint8),
             inv_gu=None, inv_dn=None, b=b, b_dn=b_dn)
    if scaled:
        d["inv_gu"] = np.exp(0.5 * rng.standard_normal((E, K))).astype(np.float32)
        d["inv_dn"] = np.exp(0.5 * rng.standard_normal((E, I))).astype(np.float32)
    return d


def on_gpu(d):
    cu = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    tile = lambda sf, K: cu(np.stack([swizzle(s, K) for s in sf]))  # noqa: E731
    K, I = d["wq_gu"].shape[2] * 2, d["wq_dn"].shape[2] * 2
    return (cu(d["wq_gu"]), tile(d["sf_gu"], K), cu(d["wq_dn"]), tile(d["sf_dn"], I)), dict(
        inv_s_gu=cu(d["inv_gu"]), inv_s_down=cu(d["inv_dn"]), had_block=d["b"], had_block_down=d["b_dn"])


def tokens(seed, T, K):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, K, generator=g)
    X[:, torch.randperm(K, generator=g)[:2]] *= 30.0
    return X.to(torch.bfloat16)


def check(X, ids, weights, d):
    """ids [T, topk] numpy (values outside the experts: dropped)."""
    E, N = d["wq_dn"].shape[:2]
    T = X.shape[0]
    off, row, pos = mq.row_groups(torch.from_numpy(ids.astype(np.int32)).cuda(), E)
    w = torch.from_numpy(weights.astype(np.float32)).cuda()
    args, kw = on_gpu(d)
    need = mq.moe_w4a16_workspace_bytes(T, ids.shape[1], E, X.shape[1], d["wq_dn"].shape[2] * 2, N)
    o, ws = Guarded(T * N * 2, dtype=torch.bfloat16, shape=(T, N)), Guarded(need)
    outs = []
    for _ in range(2):   # the second call finds what the first left in the workspace
        mq.moe_w4a16(X.cuda(), w, off, row, pos, *args, **kw, out=o.t, workspace=ws.t)
        torch.cuda.synchronize()
        assert o.intact() and ws.intact()
        outs.append(o.t.clone())
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    want, bound = opref.moe_layer(X.double().numpy(), weights.astype(np.float32).astype(np.float64), off.cpu().numpy(),
                                  row.cpu().numpy(), pos.cpu().numpy(), d)
    err = np.abs(outs[0].double().cpu().numpy() - want)
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3g} of the bound at {np.unravel_index(np.argmax(err / bound), err.shape)}"
    scale = np.linalg.norm(want)
    assert np.linalg.norm(err) <= opref.BF16 * scale + 1e-30   # rounding errors spread: their norm stays under one half step
    return outs[0]


def routing(seed, T, E, topk, drop=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(T)])
    ids[rng.random((T, topk)) < drop] = -1
    return ids, rng.random((T, topk))


@pytest.mark.parametrize("T,E,topk,K,I,N", [(1, 8, 2, 256, 128, 256), (1, 128, 8, 512, 256, 512), (3, 4, 1, 128, 128, 128),
                                            (17, 6, 3, 384, 640, 128), (64, 16, 4, 256, 256, 384), (64, 1, 1, 128, 128, 128),
                                            (33, 300, 6, 128, 128, 128), (5, 2, 2, 2048, 768, 2048), (9, 3, 2, 4224, 128, 128),
                                            (2, 3, 3, 128, 2176, 256), (8, 40, 2, 256, 384, 128), (8, 3, 2, 128, 128, 4736),
                                            (2, 4, 2, 256, 128, 4864), (16, 9, 1, 128, 256, 256), (17, 9, 1, 128, 256, 256)])
def test_sizes(T, E, topk, K, I, N):
    check(tokens(T + K, T, K), *routing(E + T, T, E, topk), layer_of(T + E + K, E, K, I, N))


@pytest.mark.parametrize("T,E,topk,K,I", [(9, 2, 2, 16384, 128), (9, 3, 1, 128, 16384), (40, 2, 1, 16384, 128), (30, 2, 2, 128, 8192),
                                          (2, 2, 1, 128, 16384), (1, 3, 3, 256, 15872)])
def test_widest_layers(T, E, topk, K, I):
    """Panels of so many channels that few rows fit: smaller chunks, and several phases per CTA."""
    check(tokens(T + K, T, K), *routing(E + T, T, E, topk), layer_of(T + E + K, E, K, I, 256))


@pytest.mark.parametrize("T,E,topk", [(4, 1024, 3), (64, 1024, 8), (64, 64, 32), (64, 32, 32), (1, 1, 1)])
def test_most_experts_and_choices(T, E, topk):
    check(tokens(T + E, T, 128), *routing(E + T, T, E, topk, drop=0.1), layer_of(T + E, E, 128, 128, 128))


@pytest.mark.parametrize("b", [1, 16, 32, 64, 128])
@pytest.mark.parametrize("b_dn", [1, 16, 32, 64, 128])
def test_hadamard_blocks(b, b_dn):
    check(tokens(b, 6, 256), *routing(b_dn, 6, 5, 2), layer_of(b + b_dn, 5, 256, 384, 128, b, b_dn, scaled=b != 32))


@pytest.mark.parametrize("T", [8, 9, 16, 17, 24, 25, 32, 33, 48, 63])
def test_all_tokens_on_one_expert(T):
    ids = np.zeros((T, 2), np.int64)
    ids[:, 0], ids[:, 1] = 2, -1
    check(tokens(T, T, 256), ids, np.random.default_rng(T).random((T, 2)), layer_of(T, 4, 256, 128, 128))


def test_dropped_choices_and_padding_rows():
    ids, w = routing(3, 20, 7, 4, drop=0.4)
    ids[5] = -1
    ids[19] = 7      # outside the experts
    out = check(tokens(1, 20, 256), ids, w, layer_of(2, 7, 256, 256, 256))
    assert bool((out[5] == 0).all()) and bool((out[19] == 0).all())
    check(tokens(1, 4, 256), np.full((4, 2), -1), np.ones((4, 2)), layer_of(2, 7, 256, 128, 128))


def test_one_expert_chosen_twice_by_a_token():
    ids = np.array([[1, 1, 0], [2, 2, 2], [0, 1, 0]])
    check(tokens(8, 3, 256), ids, np.array([[0.5, -0.25, 2.0], [1, 1, 1], [0, 0.1, 3]]), layer_of(4, 3, 256, 128, 256))


def test_every_code_and_extreme_scales():
    E, K, I, N = 2, 256, 128, 128
    d = layer_of(5, E, K, I, N, b=1, b_dn=1, scaled=False)
    d["wq_gu"] = np.tile(np.arange(256, dtype=np.uint8), (E, 2 * I, 1))[:, :, :K // 2].copy()
    d["wq_gu"][:, ::2] = d["wq_gu"][:, ::2][:, :, ::-1] ^ 0x80
    d["sf_gu"][:, :, 0] = 0      # 2^-127
    d["sf_gu"][:, :, 1] = 1
    d["sf_gu"][:, :, 2] = 252    # values up to 6 * 2^125
    d["sf_dn"][:, :, 0] = 0
    d["sf_dn"][:, :, 1] = 250
    X = torch.randn(4, K, generator=torch.Generator().manual_seed(3))
    X[:, :32] = 1.0e30
    X[:, 32:64] *= 1e-3
    X[:, 64:96] *= 1e-38
    d["wq_dn"][:, :, 16:32] = 0  # keeps the 2^123 group's products out of fp32's infinity
    check(X.to(torch.bfloat16), *routing(2, 4, E, 2), d)


def test_small_and_large_activations_share_a_token():
    """Channels 2^60 apart in different 128-blocks, and zero blocks."""
    d = layer_of(6, 3, 512, 128, 128, scaled=False)
    X = torch.randn(5, 512, generator=torch.Generator().manual_seed(1))
    X[:, :128] *= 2.0 ** -60
    X[:, 128:256] = 0.0
    X[2] = 0.0
    check(X.to(torch.bfloat16), *routing(1, 5, 3, 2), d)


def test_a_bad_token_stays_alone():
    """NaN and infinity in one token leave the others' bits as they are."""
    ids, w = routing(3, 12, 3, 2)
    d = layer_of(9, 3, 256, 128, 128)
    X = tokens(5, 12, 256)
    clean = check(X, ids, w, d)
    X[4, 7] = float("nan")
    X[6] = float("inf")
    off, row, pos = mq.row_groups(torch.from_numpy(ids.astype(np.int32)).cuda(), 3)
    args, kw = on_gpu(d)
    out = mq.moe_w4a16(X.cuda(), torch.from_numpy(w.astype(np.float32)).cuda(), off, row, pos, *args, **kw)
    torch.cuda.synchronize()
    keep = [t for t in range(12) if t not in (4, 6)]
    assert torch.equal(out[keep].view(torch.int16), clean[keep].view(torch.int16))
    assert bool(torch.isnan(out[4]).all()) and bool((~torch.isfinite(out[6].float())).all())


def test_bad_plans_stay_inside_the_buffers():
    T, E, topk = 6, 3, 2
    d = layer_of(1, E, 256, 128, 128)
    args, kw = on_gpu(d)
    X = tokens(1, T, 256).cuda()
    w = torch.ones(T, topk, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    big = 2 ** 31 - 1
    for off, row, pos in [([0, 50, -3, 7], [0, big, -1, 5, 6, 2] * 2, [[big, -1]] * T), ([-big, 4, 4, big], [0] * 12, [[0, 11]] * T),
                          ([5, 3, 12, 12], list(range(12)), [[12, 3]] * T)]:
        o = Guarded(T * 128 * 2, dtype=torch.bfloat16, shape=(T, 128))
        ws = Guarded(mq.moe_w4a16_workspace_bytes(T, topk, E, 256, 128, 128))
        mq.moe_w4a16(X, w, torch.tensor(off, **i32), torch.tensor(row, **i32), torch.tensor(pos, **i32), *args, **kw, out=o.t, workspace=ws.t)
        torch.cuda.synchronize()
        assert o.intact() and ws.intact()


def test_no_tokens():
    args, kw = on_gpu(layer_of(1, 3, 256, 128, 128))
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    n = torch.empty(0, dtype=torch.int32, device="cuda")
    assert mq.moe_w4a16(e, torch.empty(0, 2, device="cuda"), z, n, n.view(0, 2), *args, **kw).shape == (0, 128)


def test_two_graphs_and_streams_at_once():
    """Two captured layers replayed on two streams at the same time, without a shared workspace: each as when run alone."""
    d = layer_of(11, 16, 512, 256, 512)
    args, kw = on_gpu(d)
    runs = []
    for seed in (1, 2):
        ids, w = routing(seed, 32, 16, 4)
        plan = mq.row_groups(torch.from_numpy(ids.astype(np.int32)).cuda(), 16)
        X, w = tokens(seed, 32, 512).cuda(), torch.from_numpy(w.astype(np.float32)).cuda()
        alone = mq.moe_w4a16(X, w, *plan, *args, **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = mq.moe_w4a16(X, w, *plan, *args, **kw)
        runs.append((graph, out, alone, torch.cuda.Stream(), (X, w, plan)))
    for _ in range(20):
        for graph, _, _, s, _ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, alone, _, _ in runs:
        assert torch.equal(out.view(torch.int16), alone.view(torch.int16))


def test_decode_step_of_projection_adapters_router_and_experts():
    """linear_w4a16 -> lora_add -> moe_route -> moe_w4a16, eager and captured, each stage against its plain form on the
    stage's own inputs."""
    T, K, H, E, topk, L = 24, 512, 512, 16, 4, 5
    rng = np.random.default_rng(0)
    d = layer_of(21, E, H, 256, H)
    args, kw = on_gpu(d)
    X = tokens(3, T, K).cuda()
    Wq = torch.from_numpy(rng.integers(0, 256, (H, K // 2), dtype=np.uint8)).cuda()
    Wsf = torch.from_numpy(swizzle(rng.integers(116, 120, (H, K // 32), dtype=np.uint8), K)).cuda()
    g = torch.Generator("cuda").manual_seed(2)
    A = (torch.randn(L, 16, K, generator=g, device="cuda") * K ** -0.5).to(torch.bfloat16)
    B = (torch.randn(L, H, 16, generator=g, device="cuda") * 0.3).to(torch.bfloat16)
    gate = torch.randn(H, E, generator=g, device="cuda") * 0.1
    adapter = torch.randint(-1, L, (T,), generator=g, device="cuda", dtype=torch.int32)

    def step():
        y = mq.linear_w4a16(X, None, Wq, Wsf, had_block=32)
        off, row, _ = mq.row_groups(adapter, L)
        h = mq.lora_add(y, X, A, B, off, row, out=torch.empty_like(y))
        logits = h.float() @ gate
        w, ids, *plan = mq.moe_route(logits, topk)
        return y, off, row, h, logits, w, ids, *plan, mq.moe_w4a16(h, w, *plan, *args, **kw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (3, 4):
        X.copy_(tokens(seed, T, K))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)
        y, off, row, h, logits, w, ids, goff, grow, pos, out = eager
        want, bound = opref.lora(y.double(), X.double(), A.double(), B.double(), None, off.cpu(), row, opref.BF16)
        assert bool(((h.double() - want).abs() <= bound).all())
        rw, tol, rids = opref.route(logits.double().cpu().numpy(), topk, False, True, 1.0)
        np.testing.assert_array_equal(ids.cpu().numpy(), rids)
        assert np.all(np.abs(w.double().cpu().numpy() - rw) <= tol * rw)
        want, bound = opref.moe_layer(h.double().cpu().numpy(), w.double().cpu().numpy(), goff.cpu().numpy(), grow.cpu().numpy(),
                                      pos.cpu().numpy(), d)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)
