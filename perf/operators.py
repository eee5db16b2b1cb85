"""The routing, few-token mixture-of-experts and adapter operators: cases, inputs, plain forms and work.

Operators (names as the package offers them; plain forms below, in elementary torch operations):

  moe_route    logits [T, E] -> the top-k experts of every token, their weights, and the rows sorted by expert.
               A logit of -inf or NaN masks its expert; a choice that falls on a masked expert is dropped (id -1,
               weight 0, pos -1). +inf counts as the largest finite fp32. Ties go to the lowest expert.
               softmax scoring: p = softmax(logits) over the E experts; sigmoid scoring: p = 1 / (1 + exp(-logit));
               weight = scale * p, or scale * p / sum of p over the token's choices (renormalize).
  row_groups   group ids [T] or [T, topk] -> rows sorted by group, in order of entry within a group; ids outside
               [0, E) come after the last group. group_offsets [E + 1], row_index [R] (the token of every sorted
               row), pos [R] (the sorted row of every entry, -1 for the ids outside).
  moe_w4a16    a whole expert layer for few tokens, on MXFP4 weights and bf16 activations:
               g, u = gate and up rows of (x diag(inv_s) H_b) W_gu^T;  h = silu(g) u;
               y_r = (h diag(inv_s_down) H_b') W_down^T;  out[t] = sum over j of weights[t, j] y_{pos[t, j]}
  lora_add     out[m] = Y[m] + scale[a] (X[m] A[a]^T) B[a]^T for the rows m of adapter a; other rows are copied.
"""
import math

import torch

own = False

FLT_MAX = 3.4028234663852886e38


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token of a 128-expert, top-8 model: pure latency
        dict(name="route_decode_1", op="route", T=1, E=128, topk=8, dtype="bf16", scoring="softmax", renorm=True, masked=0, pad=0),
        # a prefill batch of the same model
        dict(name="route_prefill_8192", op="route", T=8192, E=128, topk=8, dtype="bf16", scoring="softmax", renorm=True, masked=0, pad=0),
        # odd sizes: fp32 logits, sigmoid scores as they are, experts masked off, and padding rows of a batch
        dict(name="route_sigmoid_odd", op="route", T=1237, E=72, topk=6, dtype="fp32", scoring="sigmoid", renorm=False, masked=9, pad=37),
        # the adapter of each request of a decode batch, some without one
        dict(name="groups_decode_64", op="groups", T=64, topk=1, E=32, absent=0.15),
        # expert choices of a prefill batch made elsewhere (a router outside this library)
        dict(name="groups_prefill_65536", op="groups", T=8192, topk=8, E=128, absent=0.0),
        # the expert layer of one decoded token (MoE 30B-A3B: hidden 2048, intermediate 768, 128 experts, top-8)
        dict(name="moe_decode_1", op="moe", T=1, E=128, topk=8, K=2048, I=768, b=32, b_down=32, s=True, pad=0),
        # the same layer for a full decode batch: nearly every expert has a row
        dict(name="moe_decode_64", op="moe", T=64, E=128, topk=8, K=2048, I=768, b=32, b_down=32, s=True, pad=0),
        # a ragged batch on a small layer: few experts with many rows each, wide Hadamard blocks, padding rows
        dict(name="moe_ragged_29", op="moe", T=29, E=12, topk=3, K=1408, I=640, b=128, b_down=64, s=False, pad=4),
        # one decoded token with an adapter on the 4096 -> 14336 up projection
        dict(name="lora_decode_1", op="lora", M=1, K=4096, N=14336, r=16, L=8, dtype="bf16", absent=0.0, order="rows", wide=0),
        # a decode batch of 64 requests over 32 adapters
        dict(name="lora_decode_64", op="lora", M=64, K=4096, N=14336, r=16, L=32, dtype="bf16", absent=0.15, order="rows", wide=0),
        # a prefill of four requests, each with its adapter, and rows without one behind them
        dict(name="lora_prefill_2048", op="lora", M=2048, K=4096, N=14336, r=64, L=4, dtype="bf16", absent=0.1, order="sorted", wide=0),
        # odd sizes: fp32 output that is a column slice of a fused projection, rank 24, rows in any order
        dict(name="lora_odd_333", op="lora", M=333, K=5120, N=1024, r=24, L=9, dtype="fp32", absent=0.3, order="rows", wide=10240),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "groups", "moe", "moe", "lora", "lora"])
    if op == "route":
        E = _log_int(rng, 2, 256)
        topk = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 8192 * 128 // max(E, 128))
        return dict(op=op, T=T, E=E, topk=topk, dtype=rng.choice(["bf16", "fp32"]), scoring=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.choice([True, False]), masked=rng.choice([0, E // 8]), pad=rng.choice([0, T // 16]))
    if op == "groups":
        topk = rng.choice([1, 2, 8])
        return dict(op=op, T=_log_int(rng, 1, 65536 // topk), topk=topk, E=_log_int(rng, 1, 256), absent=rng.choice([0.0, 0.2]))
    if op == "moe":
        E, T = _log_int(rng, 4, 128), _log_int(rng, 1, 64)
        return dict(op=op, T=T, E=E, topk=rng.randint(1, min(8, E)), K=128 * rng.randint(2, 16), I=128 * rng.randint(1, 6),
                    b=rng.choice([1, 16, 32, 64, 128]), b_down=rng.choice([1, 16, 32, 64, 128]), s=rng.choice([True, False]),
                    pad=rng.choice([0, T // 8]))
    dtype = rng.choice(["bf16", "fp32"])
    N = 8 * _log_int(rng, 32, 1792 if dtype == "bf16" else 896)
    return dict(op=op, M=_log_int(rng, 1, 2048), K=8 * _log_int(rng, 32, 512), N=N, r=8 * rng.randint(1, 8), L=_log_int(rng, 1, 48),
                dtype=dtype, absent=rng.choice([0.0, 0.25]), order=rng.choice(["rows", "sorted"]), wide=rng.choice([0, N + 8 * rng.randint(1, 64)]))


# ------------------------------------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, K):
    """bf16 activations with a few outlier channels, as a transformer's hidden states have."""
    x = _randn(g, rows, K)
    hot = torch.randperm(K, generator=g, device="cuda")[:max(1, K // 200)]
    x[:, hot] *= 30.0
    return x.to(torch.bfloat16)


def _mxfp4(g, E, N, K, gain):
    """E2M1 codes of normal values and their E8M0 scales in the 128 x 4 tiling (N, K multiples of 128). gain: the
    values' root mean square times sqrt(K), within a factor of 1.5 (scales are powers of two)."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (N * K))
    for e in range(0, E, step):
        v = _randn(g, min(step, E - e), N, K // 2, 2) * 2.0
        c = torch.bucketize(v.abs(), edges, out_int32=True) + 8 * (v < 0).to(torch.int32)
        codes[e:e + step] = (c[..., 0] + 16 * c[..., 1]).to(torch.uint8)
    mid = 127 + round(math.log2(gain / (2.0 * math.sqrt(K))))
    sf = torch.randint(mid - 1, mid + 2, (E, N * K // 32), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    return codes, sf


def _plan(ids, E):
    """Rows sorted by group, made with torch as a program without row_groups would: ids int64 [T, topk], -1 absent."""
    topk = ids.shape[1]
    key = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    pos = torch.empty_like(key)
    pos[order] = torch.arange(key.numel(), device=ids.device)
    pos = torch.where(key < E, pos, -1)
    active = torch.nonzero(counts).reshape(-1)
    return dict(group_offsets=offsets, row_index=(order // topk).to(torch.int32), pos=pos.to(torch.int32).reshape(ids.shape),
                active=active, most=int(counts.max()), live=int(counts.sum()))


def prepare(case, seed):
    g = _generator(seed)
    op, st = case["op"], dict(case=case)
    i32 = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "route":
        T, E, k = case["T"], case["E"], case["topk"]
        logits = _randn(g, T, E) * 2.0 + _randn(g, E) * 0.5
        if case["masked"]:
            logits[:, torch.randperm(E, generator=g, device="cuda")[:case["masked"]]] = -math.inf
        if case["pad"]:
            logits[T - case["pad"]:] = -math.inf
        st.update(logits=logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32),
                  weights=torch.empty(T, k, dtype=torch.float32, device="cuda"), ids=i32(T, k), group_offsets=i32(E + 1),
                  row_index=i32(T * k), pos=i32(T, k))
    elif op == "groups":
        T, k, E = case["T"], case["topk"], case["E"]
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
        ids[torch.rand(T, k, generator=g, device="cuda") < case["absent"]] = -1
        st.update(ids=ids.to(torch.int32), group_offsets=i32(E + 1), row_index=i32(T * k), pos=i32(T, k))
    elif op == "moe":
        T, E, k, K, I = case["T"], case["E"], case["topk"], case["K"], case["I"]
        score = _randn(g, T, E)
        top = torch.topk(score, k, dim=1)
        ids = top.indices
        weights = torch.softmax(top.values, dim=1)
        if case["pad"]:
            ids[T - case["pad"]:] = -1
            weights[T - case["pad"]:] = 0.0
        st.update(_plan(ids, E), weights=weights.contiguous(), X=_activations(g, T, K))
        st["wq_gu"], st["wsf_gu"] = _mxfp4(g, E, 2 * I, K, 0.5)
        st["wq_down"], st["wsf_down"] = _mxfp4(g, E, K, I, 0.5)
        st["inv_s_gu"] = torch.exp(_randn(g, E, K) * 0.3) if case["s"] else None
        st["inv_s_down"] = torch.exp(_randn(g, E, I) * 0.3) if case["s"] else None
        st["out"] = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    else:
        M, K, N, r, L = case["M"], case["K"], case["N"], case["r"], case["L"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        ids = torch.randint(0, L, (M,), generator=g, device="cuda")
        ids[torch.rand(M, generator=g, device="cuda") < case["absent"]] = L
        if case["order"] == "sorted":
            ids = torch.sort(ids).values
        Y = _randn(g, M, case["wide"] or N).to(dt)
        at = (case["wide"] - N) // 8 // 2 * 8 if case["wide"] else 0
        st.update(_plan(ids[:, None], L), X=_activations(g, M, K), Y=Y[:, at:at + N],
                  A=(_randn(g, L, r, K) / math.sqrt(K)).to(torch.bfloat16),
                  B=(_randn(g, L, N, r) * 0.1 / math.sqrt(r)).to(torch.bfloat16),
                  scale=0.5 + 1.5 * torch.rand(L, generator=g, device="cuda", dtype=torch.float32),
                  out=torch.empty(M, N, dtype=dt, device="cuda"))
    return st


# ------------------------------------------------------------------------------------------------ one pass

def run(st):
    return {"route": _route, "groups": _groups, "moe": _moe, "lora": _lora}[st["case"]["op"]](st)


def _route(st):
    c = st["case"]
    if own:
        import w4a4_mxfp4_quantized_b200 as mq
        return mq.moe_route(st["logits"], c["topk"], scoring=mq.SCORE_SOFTMAX if c["scoring"] == "softmax" else mq.SCORE_SIGMOID,
                               renormalize=c["renorm"], weights=st["weights"], ids=st["ids"], group_offsets=st["group_offsets"],
                               row_index=st["row_index"], pos=st["pos"])
    l = st["logits"].float()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=FLT_MAX)
    vals, ids = torch.sort(l, dim=1, descending=True, stable=True)
    vals, ids = vals[:, :c["topk"]], ids[:, :c["topk"]]
    live = vals > -math.inf
    top = torch.where(live[:, :1], vals[:, :1], 0.0)
    if c["scoring"] == "softmax":
        p = torch.exp(vals - top)
        total = p.sum(1, keepdim=True) if c["renorm"] else torch.exp(l - top).sum(1, keepdim=True)
    else:
        ref = top.clamp(max=0.0) if c["renorm"] else torch.zeros_like(top)
        p = torch.exp(vals.clamp(max=0.0) - ref) / (1.0 + torch.exp(-vals.abs()))
        total = p.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(top)
    weights = torch.where(live, p / total, 0.0)
    ids = torch.where(live, ids, -1)
    return (weights, ids.to(torch.int32), *_groups_plain(ids, c["E"]))


def _groups_plain(ids, E):
    topk = ids.shape[1]
    key = torch.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=key.device, dtype=key.dtype)).to(torch.int32)
    rank = torch.where(key < E, torch.arange(key.numel(), device=key.device, dtype=torch.int32), -1)
    pos = torch.empty(key.numel(), dtype=torch.int32, device=key.device)
    pos[order] = rank
    return offsets, (order // topk).to(torch.int32), pos.reshape(ids.shape)


def _groups(st):
    if own:
        import w4a4_mxfp4_quantized_b200 as mq
        return mq.row_groups(st["ids"], st["case"]["E"], group_offsets=st["group_offsets"], row_index=st["row_index"], pos=st["pos"])
    return _groups_plain(st["ids"], st["case"]["E"])


def _hadamard(b, device):
    i = torch.arange(b, device=device, dtype=torch.int32)
    v = i[:, None] & i[None, :]
    v = v ^ (v >> 4)
    v = v ^ (v >> 2)
    v = v ^ (v >> 1)
    return (1 - 2 * (v & 1)).float()


def _transform(x, b):
    return x if b == 1 else (x.reshape(*x.shape[:-1], -1, b) @ _hadamard(b, x.device)).reshape(x.shape)


def _values(codes, sf, N, K):
    """fp32 values of MXFP4 weights: codes [A, N, K/2], tiled scales [A, N K / 32]."""
    c = torch.arange(256, device=codes.device, dtype=torch.int32)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    pair = torch.stack([grid[c & 15], grid[c >> 4]], dim=1)
    scale = sf.reshape(-1, N // 128, K // 128, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1, N, K // 32, 1)
    v = pair[codes.int()].reshape(-1, N, K // 32, 32)
    return v.mul_(torch.exp2(scale.float() - 127.0)).reshape(-1, N, K)


def _slots(st, absent):
    """Rows of every active group side by side: row numbers [A, most], `absent` where a group has fewer."""
    lo, hi = st["group_offsets"][st["active"]].long(), st["group_offsets"][st["active"] + 1].long()
    r = lo[:, None] + torch.arange(st["most"], device=lo.device)
    return torch.where(r < hi[:, None], r, absent)


def _moe(st):
    c = st["case"]
    if own:
        import w4a4_mxfp4_quantized_b200 as mq
        return mq.moe_w4a16(st["X"], st["weights"], st["group_offsets"], st["row_index"], st["pos"], st["wq_gu"], st["wsf_gu"],
                               st["wq_down"], st["wsf_down"], inv_s_gu=st["inv_s_gu"], inv_s_down=st["inv_s_down"],
                               had_block=c["b"], had_block_down=c["b_down"], out=st["out"])
    T, K, I, k, act = c["T"], c["K"], c["I"], c["topk"], st["active"]
    R = T * k
    row = _slots(st, R)
    token = torch.cat([st["row_index"].long(), torch.full((1,), T, device=act.device)])[row]
    x = torch.cat([st["X"].float(), torch.zeros(1, K, device=act.device)])[token]
    if c["s"]:
        x = x * st["inv_s_gu"][act][:, None]
    gu = torch.matmul(_transform(x, c["b"]), _values(st["wq_gu"][act], st["wsf_gu"][act], 2 * I, K).transpose(1, 2))
    gu = gu.reshape(*gu.shape[:2], I // 64, 2, 64)
    g, u = gu[..., 0, :].reshape(*row.shape, I), gu[..., 1, :].reshape(*row.shape, I)
    h = g / (1.0 + torch.exp(-g)) * u
    if c["s"]:
        h = h * st["inv_s_down"][act][:, None]
    y = torch.matmul(_transform(h, c["b_down"]), _values(st["wq_down"][act], st["wsf_down"][act], K, I).transpose(1, 2))
    rows = torch.zeros(R + 1, K, device=act.device)
    rows[row.reshape(-1)] = y.reshape(-1, K)
    pos = st["pos"].long()
    picked = torch.where((pos >= 0)[..., None], rows[pos], 0.0)
    return (picked * st["weights"][..., None]).sum(1).to(torch.bfloat16)


def _lora(st):
    if own:
        import w4a4_mxfp4_quantized_b200 as mq
        return mq.lora_add(st["Y"], st["X"], st["A"], st["B"], st["group_offsets"], st["row_index"], scale=st["scale"], out=st["out"])
    c, act = st["case"], st["active"]
    M, N = c["M"], c["N"]
    row = torch.cat([st["row_index"].long(), torch.full((1,), M, device=act.device)])[_slots(st, M)]
    x = torch.cat([st["X"].float(), torch.zeros(1, c["K"], device=act.device)])[row]
    v = torch.matmul(x, st["A"][act].float().transpose(1, 2))
    d = torch.matmul(v, st["B"][act].float().transpose(1, 2)) * st["scale"][act][:, None, None]
    out = torch.cat([st["Y"].float(), torch.zeros(1, N, device=act.device)])
    out[row.reshape(-1)] += d.reshape(-1, N)
    return out[:M].to(st["Y"].dtype)


# ------------------------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["topk"]
        return {"bytes": T * E * (2 if case["dtype"] == "bf16" else 4) + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    if op == "groups":
        R = case["T"] * case["topk"]
        return {"bytes": 12 * R + 4 * (case["E"] + 1), "flops": R}
    if op == "moe":
        T, E, k, K, I = (case[n] for n in ("T", "E", "topk", "K", "I"))
        live = T - case["pad"]
        active = E * (1.0 - (1.0 - k / E) ** live)   # of uniform routing
        weights = active * 3 * I * K * 17 / 32
        scales = active * 4 * (K + I) if case["s"] else 0
        return {"bytes": weights + scales + 4 * T * K + 12 * T * k + 4 * (E + 1), "flops": 6 * live * k * I * K}
    M, K, N, r, L = (case[n] for n in ("M", "K", "N", "r", "L"))
    live = M * (1.0 - case["absent"])
    active = L * (1.0 - (1.0 - 1.0 / L) ** live)
    return {"bytes": 2 * live * K + 2 * M * N * (2 if case["dtype"] == "bf16" else 4) + active * (2 * r * (K + N) + 4) + 4 * (M + L + 1),
            "flops": 2 * live * r * (K + N)}


# ------------------------------------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "route":
        return _exact_route(case, st["logits"].cpu().double())
    if op == "groups":
        return _exact_groups(st["ids"].cpu().tolist(), case["E"])
    offsets, row_index = st["group_offsets"].tolist(), st["row_index"].tolist()
    if op == "lora":
        out = st["Y"].to(f64).clone()
        for a in range(case["L"]):
            rows = row_index[offsets[a]:offsets[a + 1]]
            if rows:
                low = torch.einsum("mk,rk->mr", st["X"][rows].to(f64), st["A"][a].to(f64))
                out[rows] += st["scale"][a].to(f64) * torch.einsum("mr,nr->mn", low, st["B"][a].to(f64))
        return out
    K, I = case["K"], case["I"]
    where = {}
    for t, row in enumerate(st["pos"].tolist()):
        for j, p in enumerate(row):
            if p >= 0:
                where[p] = (t, j)
    out = torch.zeros(case["T"], K, dtype=f64, device="cuda")
    for e in range(case["E"]):
        rows = list(range(offsets[e], offsets[e + 1]))
        if not rows:
            continue
        tokens = [where[p][0] for p in rows]
        x = st["X"][tokens].to(f64)
        if case["s"]:
            x = x * st["inv_s_gu"][e].to(f64)
        gu = _exact_rotate(x, case["b"]) @ _exact_weights(st["wq_gu"][e], st["wsf_gu"][e], 2 * I, K).T
        n = torch.arange(I, device="cuda")
        gate = gu[:, 128 * (n // 64) + n % 64]
        up = gu[:, 128 * (n // 64) + 64 + n % 64]
        h = gate * torch.sigmoid(gate) * up
        if case["s"]:
            h = h * st["inv_s_down"][e].to(f64)
        y = _exact_rotate(h, case["b_down"]) @ _exact_weights(st["wq_down"][e], st["wsf_down"][e], K, I).T
        w = torch.stack([st["weights"][where[p]] for p in rows]).to(f64)
        out.index_add_(0, torch.tensor(tokens, device="cuda"), w[:, None] * y)
    return out


def _exact_rotate(x, b):
    """Sylvester's Hadamard matrix of order b on every b neighbouring columns, by halving."""
    y = x.reshape(-1, b)
    h = 1
    while h < b:
        y = y.reshape(-1, b // (2 * h), 2, h)
        y = torch.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], dim=2).reshape(-1, b)
        h *= 2
    return y.reshape(x.shape)


def _exact_weights(codes, sf, N, K):
    k = torch.arange(K, device="cuda")
    nibble = (codes.to(torch.int64)[:, k // 2] >> (4 * (k % 2))) & 15
    e, m = (nibble >> 1) & 3, (nibble & 1).to(torch.float64)
    value = torch.where(e > 0, (1 + m / 2) * torch.pow(2.0, e.to(torch.float64) - 1), m / 2)
    value = torch.where(nibble >= 8, -value, value)
    n, c = torch.arange(N, device="cuda")[:, None], torch.arange(K // 32, device="cuda")[None]
    at = (n // 128 * (K // 128) + c // 4) * 512 + (n % 32) * 16 + n % 128 // 32 * 4 + c % 4
    return value * torch.pow(2.0, sf[at].to(torch.float64) - 127)[:, k // 32]


def _exact_route(case, logits):
    k, E = case["topk"], case["E"]
    weights, ids = [], []
    for row in logits.tolist():
        row = [-math.inf if math.isnan(v) else min(v, FLT_MAX) for v in row]
        order = sorted(range(E), key=lambda e: (-row[e], e))[:k]
        order = [e for e in order if row[e] > -math.inf]
        if case["scoring"] == "softmax":
            top = max(row)
            p = {e: math.exp(row[e] - top) for e in (order if case["renorm"] else range(E)) if row[e] > -math.inf}
            total = math.fsum(p.values())
        else:
            p = {e: 1 / (1 + math.exp(-row[e])) if row[e] > 0 else math.exp(row[e]) / (1 + math.exp(row[e])) for e in order}
            total = math.fsum(p.values()) if case["renorm"] else 1.0
        weights.append([p[e] / total for e in order] + [0.0] * (k - len(order)))
        ids.append(order + [-1] * (k - len(order)))
    return (torch.tensor(weights, dtype=torch.float64), torch.tensor(ids, dtype=torch.int32), *_exact_groups(ids, E))


def _exact_groups(ids, E):
    k, members, rest = len(ids[0]), [[] for _ in range(E)], []
    for i, e in enumerate(e for row in ids for e in row):
        (members[e] if 0 <= e < E else rest).append(i)
    pos, order, offsets = [-1] * (len(ids) * k), [], [0]
    for m in members:
        for i in m:
            pos[i] = len(order)
            order.append(i)
        offsets.append(len(order))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor([i // k for i in order + rest], dtype=torch.int32),
            torch.tensor(pos, dtype=torch.int32).reshape(len(ids), k))
