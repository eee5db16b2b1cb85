"""Adapters on small integers, where every product and sum is exact in fp32 and X A^T has up to 15 bits: the output has to be
the formula's value rounded once, bit for bit, also where Y cancels the adapter's share and nothing hides a rounding of X A^T."""
import pytest
import torch

import w4a4_mxfp4_quantized_b200 as mq
from sfutil import Guarded

pytestmark = pytest.mark.gpu


def ints(g, bound, *shape):
    return torch.randint(-bound, bound + 1, shape, generator=g, device="cuda").double()


def make(seed, M, K, N, r, L, dtype, absent=0.2):
    """|X A^T| <= 2^15 and |X A^T B^T| < 2^23 (checked), so that fp32 holds every partial sum; scales are powers of two."""
    g = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(M, generator=g, device="cuda") < absent] = L
    X, A, B = ints(g, 127, M, K), ints(g, 3, L, r, K), ints(g, 3, L, N, r)
    scale = torch.tensor([1.0, 0.5, 2.0, -1.0, 4.0], device="cuda")[torch.arange(L, device="cuda") % 5]
    delta = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for a in range(L):
        rows = torch.nonzero(ids == a).reshape(-1)
        v = X[rows] @ A[a].T
        assert rows.numel() == 0 or (v.abs().max() <= 2 ** 15 and (v.abs() @ B[a].abs().T).max() < 2 ** 21)
        delta[rows] = scale[a].double() * (v @ B[a].T)
    Y = (-delta).to(dtype)   # cancels the adapter's share but for what bf16 cannot hold
    Y[::3] = ints(g, 100, Y[::3].shape[0], N).to(dtype)
    want = (Y.double() + delta).to(dtype)
    to = lambda t: t.to(torch.bfloat16)  # noqa: E731
    return dict(X=to(X), A=to(A), B=to(B), Y=Y, scale=scale, ids=ids, want=want, L=L)


def two_launches(M, K, N, r, L, dtype):
    return mq.lora_workspace_bytes(M, r, L, mq.OUT_F32 if dtype == torch.float32 else mq.OUT_BF16, K, N) > 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 72, 104, 128])
@pytest.mark.parametrize("M", [1, 40, 1500])
def test_exact(M, r, dtype):
    c = make(M + r, M, 200, 328, r, 4, dtype)
    assert two_launches(M, 200, 328, r, 4, dtype) == (M == 1500)
    off, row, _ = mq.row_groups(c["ids"], 4)
    out = mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, scale=c["scale"], out=torch.empty_like(c["Y"]))
    torch.cuda.synchronize()
    assert torch.equal(out, c["want"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_row_has_the_same_result_in_a_small_and_a_large_call(dtype):
    """Few rows go in one launch, many in two: X A^T has the same bits in both."""
    c = make(5, 1500, 320, 264, 32, 4, dtype, absent=0.0)
    off, row, _ = mq.row_groups(c["ids"], 4)
    many = mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, scale=c["scale"], out=torch.empty_like(c["Y"]))
    for i in (0, 1, 700, 1499):
        at = slice(i, i + 1)
        off, row, _ = mq.row_groups(c["ids"][at].clone(), 4)
        one = mq.lora_add(c["Y"][at].clone(), c["X"][at].clone(), c["A"], c["B"], off, row, scale=c["scale"])
        torch.cuda.synchronize()
        assert torch.equal(one[0], many[i])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,r", [(60, 16), (1500, 16), (1500, 64), (1500, 128)])
def test_column_slices_of_wider_buffers(M, r, dtype):
    """X, Y and out as slices, each with a row stride of its own, in both launch forms: nothing beside them changes."""
    K, N, L = 136, 328, 4
    c = make(M, M, K, N, r, L, dtype)
    assert two_launches(M, K, N, r, L, dtype) == (M == 1500)
    off, row, _ = mq.row_groups(c["ids"], L)
    xw = torch.full((M, 400), float("nan"), device="cuda", dtype=torch.bfloat16)
    yw = torch.full((M, 1000), 7.0, device="cuda", dtype=dtype)
    o = Guarded(M * 752 * c["Y"].element_size(), dtype=dtype, shape=(M, 752))
    o.t.fill_(5.0)
    xw[:, 64:64 + K] = c["X"]
    yw[:, 40:40 + N] = c["Y"]
    mq.lora_add(yw[:, 40:40 + N], xw[:, 64:64 + K], c["A"], c["B"], off, row, scale=c["scale"], out=o.t[:, 16:16 + N])
    torch.cuda.synchronize()
    assert o.intact() and bool((o.t[:, :16] == 5).all()) and bool((o.t[:, 16 + N:] == 5).all())
    assert torch.equal(o.t[:, 16:16 + N], c["want"]) and torch.equal(yw[:, 40:40 + N], c["Y"])
    mq.lora_add(yw[:, 40:40 + N], xw[:, 64:64 + K], c["A"], c["B"], off, row, scale=c["scale"])   # in place
    torch.cuda.synchronize()
    assert torch.equal(yw[:, 40:40 + N], c["want"])
    assert bool((yw[:, :40] == 7).all()) and bool((yw[:, 40 + N:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,r", [(60, 24), (1500, 24), (1500, 96)])
def test_sorted_rows_without_an_index(M, r, dtype):
    c = make(M, M, 264, 328, r, 7, dtype)
    assert two_launches(M, 264, 328, r, 7, dtype) == (M == 1500)
    order = torch.sort(c["ids"], stable=True).indices
    off, _, _ = mq.row_groups(c["ids"][order].contiguous(), 7)
    Y, X, want = c["Y"][order].contiguous(), c["X"][order].contiguous(), c["want"][order]
    out = mq.lora_add(Y, X, c["A"], c["B"], off, scale=c["scale"], out=torch.empty_like(Y))
    mq.lora_add(Y, X, c["A"], c["B"], off, scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(Y, want)


def among(c, L, seed):
    """The same call with its adapters somewhere in a bank of L, whose others are NaN: they must not be read."""
    g = torch.Generator("cuda").manual_seed(seed)
    where = torch.sort(torch.randperm(L, generator=g, device="cuda")[:c["L"]]).values
    bank = {k: torch.full((L, *c[k].shape[1:]), float("nan"), dtype=c[k].dtype, device="cuda") for k in ("A", "B", "scale")}
    for k in bank:
        bank[k][where] = c[k]
    ids = torch.where(c["ids"] < c["L"], where[c["ids"].clamp(max=c["L"] - 1).long()], -1).to(torch.int32)
    return dict(c, **bank, ids=ids, L=L)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,r,L", [(1, 16, 64), (40, 16, 1024), (40, 128, 65), (300, 40, 1024), (300, 104, 200), (1500, 40, 64),
                                   (1500, 16, 64), (1500, 128, 1000), (700, 72, 64), (5000, 8, 1024), (70, 24, 32),
                                   (70, 24, 33), (1500, 24, 32), (1500, 24, 33)])
def test_few_adapters_of_a_large_bank(M, r, L, dtype):
    c = among(make(M + r, M, 200, 328, r, 4, dtype), L, r)
    off, row, _ = mq.row_groups(c["ids"], L)
    o = Guarded(c["Y"].numel() * c["Y"].element_size(), dtype=dtype, shape=c["Y"].shape)
    need = mq.lora_workspace_bytes(M, r, L, mq.OUT_F32 if dtype == torch.float32 else mq.OUT_BF16, 200, 328)
    ws = Guarded(need) if need > 0 else None
    mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, scale=c["scale"], out=o.t, workspace=ws and ws.t)
    torch.cuda.synchronize()
    assert o.intact() and (ws is None or ws.intact()) and torch.equal(o.t, c["want"])
    mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, scale=c["scale"])   # in place
    torch.cuda.synchronize()
    assert torch.equal(c["Y"], c["want"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,L,N", [(64, 64, 328), (100, 33, 328), (1500, 33, 4104), (500, 100, 4104), (1100, 64, 328), (1100, 64, 4104), (3000, 1024, 328), (3000, 70, 4104)])
def test_every_adapter_of_a_large_bank(M, L, N, dtype):
    """A handful of rows to nearly every adapter: more chunks than a round of the device, and rows of none."""
    c = make(M + L, M, 72, N, 40, L, dtype)
    off, row, _ = mq.row_groups(c["ids"], L)
    out = mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, scale=c["scale"], out=torch.empty_like(c["Y"]))
    mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(out, c["want"]) and torch.equal(c["Y"], c["want"])


@pytest.mark.parametrize("M", [40, 2000])
def test_no_row_of_a_large_bank_has_an_adapter(M):
    c = make(1, M, 72, 264, 40, 100, torch.bfloat16, absent=1.1)
    off, row, _ = mq.row_groups(c["ids"], 100)
    out = mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row, out=torch.empty_like(c["Y"]))
    before = c["Y"].clone()
    mq.lora_add(c["Y"], c["X"], c["A"], c["B"], off, row)
    torch.cuda.synchronize()
    assert torch.equal(out, before) and torch.equal(c["Y"], before)


@pytest.mark.parametrize("M", [90, 2000])
def test_malformed_plans_of_a_large_bank_stay_inside_the_buffers(M):
    """Offsets that go back and forth or leave the rows: more chunks than a sound plan can have, in both launch forms."""
    L, K, N, r = 100, 72, 264, 40
    c = make(2, M, K, N, r, L, torch.bfloat16)
    big = 2 ** 31 - 1
    for off in ([0, M] * (L // 2) + [0], [0, big, -5, M // 2] * 25 + [7], [big] * (L + 1), [-1] * (L + 1)):
        o = Guarded(M * N * 2, dtype=torch.bfloat16, shape=(M, N))
        need = mq.lora_workspace_bytes(M, r, L, mq.OUT_BF16, K, N)
        ws = Guarded(need) if need > 0 else None
        mq.lora_add(c["Y"], c["X"], c["A"], c["B"], torch.tensor(off, dtype=torch.int32, device="cuda"), out=o.t, workspace=ws and ws.t)
        torch.cuda.synchronize()
        assert o.intact() and (ws is None or ws.intact())


@pytest.mark.parametrize("M,r,L", [(40, 16, 4), (40, 16, 100), (1500, 40, 4), (1500, 40, 100)])
def test_captured_once_and_replayed_with_other_plans(M, r, L):
    """Router and adapters in one graph, two of them at once on two streams: the next replay has other adapters for the rows."""
    runs = []
    for seed in (1, 2):
        first, second = (among(make(10 * seed + k, M, 136, 328, r, 4, torch.bfloat16), L, 7) for k in (0, 1))
        Y, X, ids, A, B, scale = (first[k].clone() for k in ("Y", "X", "ids", "A", "B", "scale"))

        def step():
            off, row, _ = mq.row_groups(ids, L)
            return mq.lora_add(Y, X, A, B, off, row, scale=scale, out=torch.empty_like(Y))

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((graph, out, first, second, (Y, X, ids, A, B, scale), torch.cuda.Stream()))
    for turn in (2, 3, 2):
        for graph, out, *cs, now, stream in runs:
            c = cs[turn - 2]
            for t, k in zip(now, ("Y", "X", "ids", "A", "B", "scale")):
                t.copy_(c[k])
        torch.cuda.synchronize()
        for _ in range(5):
            for run in runs:
                with torch.cuda.stream(run[-1]):
                    run[0].replay()
        torch.cuda.synchronize()
        for run in runs:
            assert torch.equal(run[1], run[turn]["want"])
