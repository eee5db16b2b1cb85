"""GPU parity of the adapters: out = Y + scale (X A^T) B^T by rows, against the plain 64-bit form within fp32 sums and one
rounding to the output type; in place and apart, strided, ragged groups, rows of no adapter, every rank."""
import pytest
import torch

import opref
import w4a4_mxfp4_quantized_b200 as mq
from sfutil import Guarded

pytestmark = pytest.mark.gpu


def make(seed, M, K, N, r, L, dtype, absent=0.2):
    g = torch.Generator("cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(M, generator=g, device="cuda") < absent] = -1
    return dict(Y=rn(M, N).to(dtype), X=rn(M, K).to(torch.bfloat16), A=(rn(L, r, K) * K ** -0.5).to(torch.bfloat16),
                B=rn(L, N, r).to(torch.bfloat16), scale=rn(L), ids=ids)


def reference(Y, X, A, B, scale, off, row):
    f = lambda t: None if t is None else t.double()  # noqa: E731
    return opref.lora(f(Y), f(X), f(A), f(B), f(scale), off.cpu(), row, torch.finfo(Y.dtype).eps / 2)


def check(c, in_place=False, scaled=True, sort=False):
    L = c["A"].shape[0]
    if sort:
        c["ids"] = torch.sort(torch.where(c["ids"] < 0, L, c["ids"])).values.to(torch.int32)
    off, row, _ = mq.row_groups(c["ids"], L)
    scale = c["scale"] if scaled else None
    Y = c["Y"]
    want, bound = reference(Y, c["X"], c["A"], c["B"], scale, off, row)
    o = Guarded(Y.numel() * Y.element_size(), dtype=Y.dtype, shape=Y.shape)
    if in_place:
        o.t.copy_(Y)
    got = mq.lora_add(o.t if in_place else Y, c["X"], c["A"], c["B"], off, None if sort else row, scale=scale,
                      out=None if in_place else o.t)
    torch.cuda.synchronize()
    assert o.intact() and got.data_ptr() == o.t.data_ptr()
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    rest = row[int(off[-1]):].long()
    assert torch.equal(got[rest], Y[rest])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N,r,L", [(1, 4096, 1024, 16, 1), (7, 256, 512, 8, 3), (64, 2048, 1536, 16, 40), (333, 1000, 776, 24, 5),
                                       (130, 8, 8, 8, 2), (2050, 512, 264, 64, 3), (1, 136, 4104, 128, 2), (50, 1288, 1032, 104, 6),
                                       (17, 640, 8200, 40, 1024)])
def test_sizes(M, K, N, r, L, dtype):
    check(make(M + K + N, M, K, N, r, L, dtype))


@pytest.mark.parametrize("r", [8, 16, 32, 48, 64, 72, 96, 128])
def test_ranks_in_place(r):
    check(make(r, 90, 384, 640, r, 4, torch.bfloat16), in_place=True, scaled=False)


@pytest.mark.parametrize("M", [1, 16, 17, 64, 127, 128, 129, 1000])
def test_rows_of_one_adapter(M):
    check(make(M, M, 512, 512, 16, 1, torch.bfloat16, absent=0.0), in_place=True)


def test_sorted_rows_need_no_index():
    check(make(1, 500, 256, 384, 16, 7, torch.float32), sort=True)


def test_no_row_and_every_row_without_adapter():
    c = make(2, 40, 256, 256, 16, 3, torch.bfloat16, absent=1.1)
    check(c)
    check(c, in_place=True)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert mq.lora_add(e, e, c["A"], c["B"], off).shape == (0, 256)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_column_slices(dtype):
    """Y, out and X as column slices of wider buffers: nothing beside the slice changes."""
    c = make(6, 100, 264, 520, 16, 4, dtype)
    off, row, _ = mq.row_groups(c["ids"], 4)
    g = torch.Generator("cuda").manual_seed(0)
    wide = torch.randn(100, 1600, generator=g, device="cuda").to(dtype)
    xw = torch.randn(100, 800, generator=g, device="cuda").to(torch.bfloat16)
    Y, X = wide[:, 640:640 + 520], xw[:, 16:16 + 264]
    before = wide.clone()
    want, bound = reference(Y, X, c["A"], c["B"], c["scale"], off, row)
    apart = torch.zeros(100, 1040, device="cuda", dtype=dtype)
    mq.lora_add(Y, X, c["A"], c["B"], off, row, scale=c["scale"], out=apart[:, 8:528])
    torch.cuda.synchronize()
    assert torch.equal(wide, before) and bool((apart[:, :8] == 0).all()) and bool((apart[:, 528:] == 0).all())
    mq.lora_add(Y, X, c["A"], c["B"], off, row, scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(wide[:, :640], before[:, :640]) and torch.equal(wide[:, 1160:], before[:, 1160:])
    assert torch.equal(Y, apart[:, 8:528])
    assert bool(((Y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("M,dtype", [(64, torch.float32), (300, torch.bfloat16), (1500, torch.float32), (1500, torch.bfloat16)])
def test_values_of_other_rows_and_adapters_do_not_leak(M, dtype):
    """NaN and infinities in one row of X, and in one adapter's A, stay in that row and that adapter's rows."""
    c = make(3, M, 256, 256, 24, 4, dtype, absent=0.0)
    c["X"][5] = float("nan")
    c["X"][6, 3] = float("inf")
    c["A"][2, 4] = float("nan")
    off, row, _ = mq.row_groups(c["ids"], 4)
    out = mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, out=torch.empty_like(c["Y"]))
    torch.cuda.synchronize()
    hit = (c["ids"] == 2)
    hit[5] = hit[6] = True
    assert bool(torch.isfinite(out[~hit]).all())
    assert bool(torch.isnan(out[5]).all()) and bool((~torch.isfinite(out[6])).all())


def test_bad_plans_stay_inside_the_buffers():
    c = make(4, 30, 256, 256, 16, 3, torch.bfloat16)
    off = torch.tensor([0, 90, -7, 12], dtype=torch.int32, device="cuda")
    row = torch.arange(30, dtype=torch.int32, device="cuda")
    row[4], row[9] = -3, 2 ** 31 - 1
    o = Guarded(c["Y"].numel() * 2, dtype=torch.bfloat16, shape=c["Y"].shape)
    mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, out=o.t)
    torch.cuda.synchronize()
    assert o.intact()


def test_overlapping_groups_in_two_launches_stay_inside_the_workspace():
    """Offsets that go back and forth: more chunks than a sound plan of so many rows can have."""
    M, N, L = 600, 4096, 16
    c = make(5, M, 128, N, 64, L, torch.bfloat16)
    off = torch.tensor([0, M] * (L // 2) + [0], dtype=torch.int32, device="cuda")
    y, ws = Guarded(M * N * 2, dtype=torch.bfloat16, shape=(M, N)), Guarded(mq.lora_workspace_bytes(M, 64, L, K=128, N=N))
    mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, out=y.t, workspace=ws.t)
    torch.cuda.synchronize()
    assert y.intact() and ws.intact()


def test_an_infinity_stays_one():
    """X A^T beyond the parts' range: the output is the infinity that the formula gives, not NaN."""
    for M, dtype in ((3, torch.bfloat16), (3, torch.float32), (200, torch.bfloat16), (1500, torch.float32)):
        A = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda")
        A[0, :, 0] = 1.0
        X = torch.zeros(M, 64, dtype=torch.bfloat16, device="cuda")
        X[1, 0] = float("inf")
        B = torch.ones(1, 40, 8, dtype=torch.bfloat16, device="cuda")
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        out = mq.lora_add(torch.zeros(M, 40, dtype=dtype, device="cuda"), X, A, B, off)
        torch.cuda.synchronize()
        assert bool(torch.isinf(out[1]).all()) and bool((out[0] == 0).all()), (M, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r", [8, 40, 64, 72, 128])
def test_many_rows_in_two_launches(r, dtype):
    """Enough rows for the two-launch form: in place and apart, with its workspace guarded."""
    c = make(r, 1300, 320, 328, r, 3, dtype)
    off, row, _ = mq.row_groups(c["ids"], 3)
    need = mq.lora_workspace_bytes(1300, r, 3, mq.OUT_F32 if dtype == torch.float32 else mq.OUT_BF16)
    assert need > 0
    want, bound = reference(c["Y"], c["X"], c["A"], c["B"], c["scale"], off, row)
    ws, y = Guarded(need), Guarded(c["Y"].numel() * c["Y"].element_size(), dtype=dtype, shape=c["Y"].shape)
    y.t.copy_(c["Y"])
    apart = mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, scale=c["scale"], out=torch.empty_like(c["Y"]), workspace=ws.t)
    mq.lora_add(y.t, c["X"], c["A"], c["B"], off, row, scale=c["scale"], workspace=ws.t)
    torch.cuda.synchronize()
    assert ws.intact() and y.intact() and torch.equal(apart, y.t)
    assert bool(((apart.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N,r,L", [(16, 72, 40008, 128, 1), (33, 520, 40000, 64, 2), (65, 8, 90008, 24, 1), (100, 4104, 10008, 96, 3)])
def test_two_launches_for_few_rows_on_many_columns(M, K, N, r, L, dtype):
    assert mq.lora_workspace_bytes(M, r, L, mq.OUT_BF16, K, N) > 0
    check(make(M, M, K, N, r, L, dtype))


@pytest.mark.parametrize("M", [2100, 4100, 8200, 20100])
@pytest.mark.parametrize("K,r", [(72, 8), (584, 64)])
def test_clusters_of_eight_to_one(M, K, r):
    """Fewer CTAs per chunk as the chunks grow in number; K narrower than all of them take, and with a ragged end."""
    check(make(M, M, K, 136, r, 3, torch.bfloat16))


def test_two_calls_at_once():
    """The two-launch form on two streams at the same time, each with its own workspace."""
    cs = [make(s, 1500, 512, 1024, 16, 4, torch.bfloat16) for s in (1, 2)]
    plans = [mq.row_groups(c["ids"], 4)[:2] for c in cs]
    alone = [mq.lora_add(c["Y"], c["X"], c["A"], c["B"], *p, out=torch.empty_like(c["Y"])) for c, p in zip(cs, plans)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in cs], [torch.empty_like(c["Y"]) for c in cs]
    for _ in range(10):
        for c, p, s, o in zip(cs, plans, streams, outs):
            with torch.cuda.stream(s):
                mq.lora_add(c["Y"], c["X"], c["A"], c["B"], *p, out=o)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert torch.equal(a, o)


@pytest.mark.parametrize("M", [64, 1500])
def test_captured_graph_and_other_stream_agree(M):
    c = make(7, M, 1024, 768, 16, 9, torch.bfloat16)
    off, row, _ = mq.row_groups(c["ids"], 9)
    args = (c["Y"], c["X"], c["A"], c["B"], off, row)
    want = mq.lora_add(*args, scale=c["scale"], out=torch.empty_like(c["Y"]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = mq.lora_add(*args, scale=c["scale"], out=torch.empty_like(c["Y"]))
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(c["Y"])
    with torch.cuda.graph(graph):
        mq.lora_add(*args, scale=c["scale"], out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, other) and torch.equal(want, out)
