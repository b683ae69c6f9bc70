"""The rest of a layer between the re-layouts as it is measured: attention with a
sliding window and sinks on head shards, layer norm on sequence shards, and the
balance loss of a router, each with its gradient.

``run`` computes each operator in plain torch operations (``own`` false) or
through the library's entry points (``own`` true), on what ``prepare`` made.
``exact`` computes the same from the definitions in 64 bits.

Definitions.

  attend       Sequence b has lengths[b] tokens in a cache of S; its query i
               stands at position p = starts[b] + i.  It sees the keys j <= p with
               p - j < window or j < sinks, and none if p is outside
               [0, lengths[b]).  o = softmax(scale * q k) v over the visible
               keys, lse the logarithm of the softmax's sum; 0 and -inf where a
               row sees nothing.  Query head h reads key head h / (Hq / Hkv).
  attend_grad  the same, and the gradients of q, k, v for a gradient of o
  attend_step  the same for the last tokens of sequences in a long cache
  norm         y = (x - mean) * rstd * weight + bias per row, mean, rstd =
               1 / sqrt(variance + eps)
  norm_grad    gradients of x, weight and bias
  balance      p = softmax(logits) per token; counts[e]: choices of e by live
               tokens; with L live tokens f[e] = E * counts[e] / (K * L), loss =
               coef * sum_e f[e] * mean over live t of p[t, e]; slope = coef * f / L
  balance_grad the same, and the gradient of the logits (counts are constants)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
COEF = 0.01


def listed():
    return [
        # one new token for each of 16 sequences, 1024 tokens of a 4096 token cache in sight: the call's latency counts
        dict(name="step_window", op="attend_step", N=8, B=16, groups=1, S=4096, Hq=32, Hkv=8, d=64, queries=1,
             window=1024, sinks=4, layout="head", padded=True, dtype="bf16"),
        # few long sequences, the whole cache in sight: bound by reading it
        dict(name="step_long", op="attend_step", N=8, B=4, groups=1, S=65536, Hq=32, Hkv=8, d=128, queries=1,
             window=65536, sinks=0, layout="head", padded=True, dtype="fp16"),
        # the forward pass of two 16k sequences over eight ranks
        dict(name="attend_train", op="attend", N=8, B=2, groups=2, S=16384, Hq=32, Hkv=8, d=64, queries=16384,
             window=1024, sinks=4, layout="head", padded=False, dtype="bf16"),
        # a training step of a short, padded batch in full precision: odd sizes, three query heads a key head
        dict(name="attend_grad_odd", op="attend_grad", N=2, B=3, groups=1, S=998, Hq=12, Hkv=4, d=40, queries=998,
             window=201, sinks=3, layout="token", padded=True, dtype="fp32"),
        # the largest: a training step of two 8k sequences with heads of 128 channels
        dict(name="attend_grad_train", op="attend_grad", N=8, B=2, groups=2, S=8192, Hq=32, Hkv=8, d=128, queries=8192,
             window=2048, sinks=16, layout="head", padded=False, dtype="bf16"),
        # a small serving batch
        dict(name="norm_decode", op="norm", T=16, D=4096, dtype="bf16", weight="bf16"),
        # a micro-batch of two 16k sequences
        dict(name="norm_train", op="norm", T=32768, D=4096, dtype="bf16", weight="fp32"),
        # an odd width in full precision
        dict(name="norm_grad_odd", op="norm_grad", T=4099, D=777, dtype="fp32", weight="fp32"),
        # both gradients of a micro-batch
        dict(name="norm_grad_train", op="norm_grad", T=32768, D=2048, dtype="bf16", weight="fp32"),
        # a small batch with padding
        dict(name="balance_small", op="balance", T=250, K=2, E=8, padded=True, dtype="fp32", id_bytes=8),
        # a router's micro-batch
        dict(name="balance_train", op="balance", T=32768, K=8, E=128, padded=False, dtype="fp32", id_bytes=8),
        # and with its gradient, 16 bit scores and many experts
        dict(name="balance_grad_train", op="balance_grad", T=32768, K=4, E=320, padded=True, dtype="bf16", id_bytes=4),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["attend", "attend_grad", "attend_step", "norm", "norm_grad", "balance", "balance_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    while True:
        if op.startswith("attend"):
            groups, members = rng.choice([1, 1, 2]), rng.choice([1, 2, 4])
            kv = rng.choice([1, 2, 4])
            case = dict(op=op, N=groups * members, groups=groups, Hkv=members * kv,
                        Hq=members * kv * rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 64, 128, 128, 80, 40, 96, 20]))
            if op == "attend_step":
                case.update(B=groups * _log(rng, 1, 16), S=members * _log(rng, 16, 32768 // members), queries=rng.choice([1, 1, 1, 2, 5]))
            else:
                S = members * _log(rng, 2, 16384 // members)
                case.update(B=groups * rng.choice([1, 1, 2, 3]), S=S, queries=S)
            case["queries"] = min(case["queries"], case["S"])
            case["window"] = rng.choice([case["S"], _log(rng, 2, 4096)])
            case.update(sinks=rng.choice([0, 1, 4, 16, 70]), layout=rng.choice(["head", "head", "token"]),
                        padded=op == "attend_step" or rng.random() < 0.5, dtype=dtype)
            blocks = _blocks(case)
            pairs = case["B"] * case["Hq"] * blocks[0] * blocks[1] * (blocks[1] + min(case["S"], case["window"]))
            w = work(case)
            # fp32 products run at a sixteenth of the 16 bit rate
            if pairs <= 2.2e9 and w["flops"] * (16 if dtype == "fp32" else 1) <= 1.6e12 and w["bytes"] <= 1.1e9:
                return case
        elif op.startswith("norm"):
            D = _log(rng, 32, 12288)
            case = dict(op=op, T=_log(rng, 1, 65536), D=D // 64 * 64 if D >= 64 and rng.random() < 0.6 else D, dtype=dtype,
                        weight=rng.choice([dtype, "fp32"]))
            if work(case)["bytes"] <= 5.4e8:
                return case
        else:
            # fewer choices than experts, or all counts are the same
            E = _log(rng, 4, 1024)
            return dict(op=op, T=_log(rng, 16, 32768), K=rng.randint(1, min(8, E - 1)), E=E, padded=rng.random() < 0.5, dtype=dtype,
                        id_bytes=rng.choice([4, 8]))


# ------------------------------------------------------------------ inputs --

def _shards(case):
    """(rank, sequence) pairs of the head-sharded buffers, query and key heads of each."""
    P = case["N"] // case["groups"]
    return case["B"] * P, case["Hq"] // P, case["Hkv"] // P


def _sequence_of(case, device):
    """The sequence of each shard, in the order of the buffers."""
    P, Bl = case["N"] // case["groups"], case["B"] // case["groups"]
    n = torch.arange(case["B"] * P, device=device)
    return n // Bl // P * Bl + n % Bl


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(dt)

    state = dict(case=case)
    if case["op"].startswith("attend"):
        shards, hq, hkv = _shards(case)
        B, S, d, queries = case["B"], case["S"], case["d"], case["queries"]
        nq, nkv = shards * hq * queries * d, shards * hkv * S * d
        lengths = torch.full((B,), S, dtype=torch.int32, device=dev)
        if case["padded"]:
            # the longest fills the cache, the others end anywhere in its last three quarters
            lengths = (S - (torch.rand(B, generator=g, device=dev) * 0.75 * S).int()).int()
            lengths[0] = S
        state.update(lengths=lengths, starts=lengths - queries if case["op"] == "attend_step" else torch.zeros_like(lengths),
                     scale=d ** -0.5)
        qkv = normal(nq + 2 * nkv)
        state.update(q=qkv[:nq], k=qkv[nq:nq + nkv], v=qkv[nq + nkv:], o=torch.empty(nq, dtype=dt, device=dev),
                     lse=torch.empty(nq // d, device=dev))
        if case["op"] == "attend_grad":
            dqkv = torch.empty_like(qkv)
            state.update(do=normal(nq), dq=dqkv[:nq], dk=dqkv[nq:nq + nkv], dv=dqkv[nq + nkv:])
    elif case["op"].startswith("norm"):
        T, D, wt = case["T"], case["D"], DTYPES[case["weight"]]
        # rows of different size about different means, as a residual stream has them
        x = torch.randn(T, D, generator=g, device=dev) * torch.exp(torch.randn(T, 1, generator=g, device=dev) * 0.5)
        x = (x + torch.randn(T, 1, generator=g, device=dev)).to(dt)
        state.update(x=x, weight=(1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(wt),
                     bias=(0.1 * torch.randn(D, generator=g, device=dev)).to(wt))
        if case["op"] == "norm":
            state.update(y=torch.empty_like(x), mean=torch.empty(T, device=dev), rstd=torch.empty(T, device=dev))
        else:
            mean, rstd = _statistics(x)
            state.update(dy=normal(T, D), mean=mean.view(T), rstd=rstd.view(T), dx=torch.empty_like(x),
                         dweight=torch.empty(D, dtype=wt, device=dev), dbias=torch.empty(D, dtype=wt, device=dev))
    else:
        T, K, E = case["T"], case["K"], case["E"]
        logits = normal(T, E) + (0.5 * torch.randn(E, generator=g, device=dev)).to(dt)
        ids = torch.topk(logits.float(), K, dim=1).indices.to(torch.int32 if case["id_bytes"] == 4 else torch.int64)
        mask = torch.ones(T, dtype=torch.uint8, device=dev)
        if case["padded"]:
            mask = (torch.rand(T, generator=g, device=dev) < 0.8).to(torch.uint8)
            mask[0] = 1
        state.update(logits=logits, ids=ids.contiguous(), mask=mask, dloss=torch.rand(1, generator=g, device=dev) + 0.5,
                     loss=torch.empty(1, device=dev), counts=torch.empty(E, dtype=torch.int32, device=dev),
                     slope=torch.empty(E, device=dev), dlogits=torch.empty_like(logits))
    if own:
        state.update(_plan(case))
    return state


def _plan(case):
    """The plan and the workspaces that a program keeps for its sizes."""
    from sequence_re_layout_amd import binding as b
    code = {"bf16": b.BASP_BF16, "fp16": b.BASP_FP16, "fp32": b.BASP_FP32}
    dt = code[case["dtype"]]
    if case["op"].startswith("attend"):
        order = b.BASP_LAYOUT_HEAD_MAJOR if case["layout"] == "head" else b.BASP_LAYOUT_TOKEN_MAJOR
        layout = b.basp_plan_create_groups(case["N"], case["B"], case["S"], case["Hq"], case["Hkv"], case["d"], dt,
                                           case["groups"], order)
        plan = b.basp_attention_plan_create(layout, case["queries"], case["window"], case["sinks"])
        need = plan.info["grad_workspace_bytes" if case["op"] == "attend_grad" else "workspace_bytes"]
        if case["op"] == "attend_grad":
            need = max(need, plan.info["workspace_bytes"])
    elif case["op"].startswith("norm"):
        plan = b.basp_norm_plan_create(case["T"], case["D"], dt, code[case["weight"]])
        need = plan.info["workspace_bytes"]
    else:
        plan = b.basp_expert_plan_create(case["T"], case["K"], case["E"], 1, id_bytes=case["id_bytes"], weight_dtype=dt)
        need = b.basp_balance_workspace_bytes(plan)
    return dict(b=b, plan=plan, ws=torch.empty(max(1, need), dtype=torch.uint8, device="cuda"))


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        b, plan = s["b"], s["plan"]
        if op.startswith("attend"):
            step = op == "attend_step"
            b.basp_attention(plan, s["q"], s["k"], s["v"], s["starts"], s["lengths"], s["scale"], s["o"],
                             None if step else s["lse"], s["ws"])
            if step:
                return s["o"]
            if op == "attend":
                return s["o"], s["lse"]
            b.basp_attention_grad(plan, s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["starts"], s["lengths"],
                                  s["scale"], s["dq"], s["dk"], s["dv"], s["ws"])
            return s["o"], s["lse"], s["dq"], s["dk"], s["dv"]
        if op == "norm":
            b.basp_layer_norm(plan, s["x"], s["weight"], s["bias"], EPS, s["y"], s["mean"], s["rstd"])
            return s["y"], s["mean"], s["rstd"]
        if op == "norm_grad":
            b.basp_layer_norm_grad(plan, s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                                   s["ws"])
            return s["dx"], s["dweight"], s["dbias"]
        b.basp_balance_loss(plan, s["logits"], s["ids"], s["mask"], COEF, s["loss"], s["counts"], s["slope"], s["ws"])
        if op == "balance":
            return s["loss"], s["counts"], s["slope"]
        b.basp_balance_loss_grad(plan, s["logits"], s["mask"], s["slope"], s["dloss"], s["dlogits"])
        return s["loss"], s["counts"], s["slope"], s["dlogits"]
    return _PLAIN[op](s["case"], s)


# -------------------------------------------------------------- plain form --

def _blocks(case):
    """Query blocks and their length: a block's queries are multiplied with all keys that one of them may see."""
    queries = case["queries"]
    if case["window"] >= case["S"]:
        return 1, queries
    c = max(1, min(queries, case["window"]))
    return (queries + c - 1) // c, c


def _heads(case, x, heads, tokens):
    """A head-sharded buffer as [shards][tokens][heads][d]."""
    shards, d = _shards(case)[0], case["d"]
    if case["layout"] == "head":
        return x.view(shards, heads, tokens, d).transpose(1, 2)
    return x.view(shards, tokens, heads, d)


def _buffer(case, x):
    """[shards][tokens][heads][d] as a head-sharded buffer."""
    return (x.transpose(1, 2) if case["layout"] == "head" else x).reshape(-1)


def _plain_attend(case, s):
    shards, hq, hkv = _shards(case)
    S, d, queries, window, sinks = case["S"], case["d"], case["queries"], case["window"], case["sinks"]
    dev, ratio = s["q"].device, hq // hkv
    n, C = _blocks(case)
    seq = _sequence_of(case, dev)
    starts, lengths = s["starts"].long()[seq], s["lengths"].long()[seq]
    # the keys that each block is multiplied with: the sinks, and those from its first query's window on
    if window >= S:
        sinks, first = 0, torch.zeros(shards, 1, dtype=torch.long, device=dev)
        width = S
    else:
        first = starts[:, None] + torch.arange(n, device=dev) * C - window + 1
        width = C + window - 1
    band = first[:, :, None] + torch.arange(width, device=dev)
    key = torch.cat([torch.arange(sinks, device=dev).expand(shards, n, sinks), band], 2)
    there = torch.cat([torch.ones(shards, n, sinks, dtype=torch.bool, device=dev), band >= sinks], 2)
    row = torch.arange(n * C, device=dev)
    at = (starts[:, None] + row).view(shards, n, C, 1)
    j = key[:, :, None, :]
    sees = there[:, :, None, :] & (j >= 0) & (j <= at) & (at < lengths[:, None, None, None]) & (
        (at - j < window) | (j < sinks)) & (at >= 0) & (row.view(n, C, 1) < queries)
    key = key.clamp(0, S - 1)
    shard = torch.arange(shards, device=dev)[:, None, None]

    def blocks(x):                   # [shards][Hkv][n][ratio * C][d], query rows by head of a group and position
        x = x[:, row.clamp(max=queries - 1)].float()
        return x.view(shards, n, C, hkv, ratio, d).permute(0, 3, 1, 4, 2, 5).reshape(shards, hkv, n, ratio * C, d)

    def keys(x):                     # [shards][Hkv][n][keys][d]
        x = x[shard, key].float().masked_fill_(~there[..., None, None] | (key >= lengths[:, None, None])[..., None, None], 0.0)
        return x.permute(0, 3, 1, 2, 4).contiguous()

    def back(x):                     # the queries' rows as a buffer
        x = x.view(shards, hkv, n, ratio, C, -1).permute(0, 2, 4, 1, 3, 5).reshape(shards, n * C, hq, -1)
        return x[:, :queries]

    q, k, v = blocks(_heads(case, s["q"], hq, queries)), keys(_heads(case, s["k"], hkv, S)), keys(_heads(case, s["v"], hkv, S))
    hidden = ~sees[:, None, :, None]                                          # [shards][1][n][1][C][keys]
    p = (q @ k.transpose(3, 4) * s["scale"]).view(shards, hkv, n, ratio, C, -1).masked_fill_(hidden, -math.inf)
    most = p.amax(5, keepdim=True)
    most = torch.where(most == -math.inf, torch.zeros_like(most), most)
    p = (p - most).exp_()
    total = p.sum(5, keepdim=True)
    lse = back(total.log() + most)[..., 0]
    p = (p / torch.where(total == 0, torch.ones_like(total), total)).view(shards, hkv, n, ratio * C, -1)
    o = p @ v
    dt = s["q"].dtype
    out = _buffer(case, back(o)).to(dt)
    lse = lse.transpose(1, 2).reshape(-1)
    if case["op"] == "attend_step":
        return out
    if case["op"] == "attend":
        return out, lse
    do = blocks(_heads(case, s["do"], hq, queries))
    live = sees.any(3)[:, None, :, None].expand(shards, 1, n, ratio, C).reshape(shards, 1, n, ratio * C, 1)
    do = do.masked_fill_(~live, 0.0)
    dv = p.transpose(3, 4) @ do
    ds = do @ v.transpose(3, 4)
    ds = (ds - (ds * p).sum(4, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = _buffer(case, back(ds @ k)).to(dt)
    dk = ds.transpose(3, 4) @ q
    flat = (shard * S + key).reshape(-1)

    def gathered(x):                 # sums over the blocks that a key belongs to
        x = x.permute(0, 2, 3, 1, 4).reshape(-1, hkv * d)
        return _buffer(case, torch.zeros(shards * S, hkv * d, device=dev).index_add_(0, flat, x).view(shards, S, hkv, d)).to(dt)

    return out, lse, dq, gathered(dk), gathered(dv)


def _statistics(x):
    f = x.float()
    mean = f.mean(1, keepdim=True)
    return mean, 1.0 / torch.sqrt((f - mean).square().mean(1, keepdim=True) + EPS)


def _plain_norm(case, s):
    mean, rstd = _statistics(s["x"])
    y = (s["x"].float() - mean) * rstd * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_norm_grad(case, s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    wt = s["weight"].dtype
    return dx.to(s["x"].dtype), (dy * xhat).sum(0).to(wt), dy.sum(0).to(wt)


def _plain_balance(case, s):
    T, K, E = case["T"], case["K"], case["E"]
    live = s["mask"] != 0
    x = s["logits"].float()
    p = (x - x.amax(1, keepdim=True)).exp_()
    p = (p / p.sum(1, keepdim=True)).masked_fill_(~live[:, None], 0.0)
    L = live.sum()
    kept = live[:, None].expand(T, K).reshape(-1).long()
    counts = torch.zeros(E, dtype=torch.long, device=x.device).scatter_add_(0, s["ids"].reshape(-1).long(), kept)
    f = counts.float() * E / (K * L)
    loss = COEF * (f * p.sum(0)).sum() / L
    slope = COEF * f / L
    if case["op"] == "balance":
        return loss.view(1), counts.int(), slope
    dlogits = s["dloss"] * p * (slope - (p * slope).sum(1, keepdim=True))
    return loss.view(1), counts.int(), slope, dlogits.to(s["logits"].dtype)


_PLAIN = {"attend": _plain_attend, "attend_grad": _plain_attend, "attend_step": _plain_attend, "norm": _plain_norm,
          "norm_grad": _plain_norm_grad, "balance": _plain_balance, "balance_grad": _plain_balance}


def _seen(length, first, queries, window, sinks):
    """Visible (query, key) pairs of one head."""
    total = 0
    lo, hi = max(first, 0), min(first + queries, length)
    if hi <= lo:
        return 0
    # positions up to window - 1 see all before them, later ones the window and the sinks outside it
    mid = min(max(lo, window), hi)
    total += (lo + 1 + mid) * (mid - lo) // 2
    total += window * (hi - mid)
    a, z = mid - window + 1, hi - window + 1        # keys before the window of these positions
    if z > a:
        n = min(max(sinks - a, 0), z - a)
        total += (a + a + n - 1) * n // 2 + sinks * (z - a - n)
    return total


def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    if case["op"].startswith("attend"):
        B, S, d, queries, window, sinks = (case[n] for n in ("B", "S", "d", "queries", "window", "sinks"))
        mean = int(S * 0.625) if case["padded"] else S
        of = [S] + [mean] * (B - 1)
        firsts = [n - queries for n in of] if case["op"] == "attend_step" else [0] * B
        pairs = sum(_seen(n, f, queries, window, sinks) for n, f in zip(of, firsts)) * case["Hq"]
        # tokens whose keys and values some query sees
        used = sum(min(n, min(window - 1, max(n, 0)) + queries + sinks) if case["op"] == "attend_step" else n for n in of)
        rows = B * queries * case["Hq"]
        bytes_ = (2 * rows * d + 2 * used * case["Hkv"] * d) * es
        if case["op"] != "attend_step":
            bytes_ += rows * 4
        if case["op"] != "attend_grad":
            return {"bytes": bytes_, "flops": 4 * d * pairs}
        return {"bytes": bytes_ + (2 * rows * d + 2 * B * S * case["Hkv"] * d) * es, "flops": 14 * d * pairs}
    if case["op"].startswith("norm"):
        T, D, ws = case["T"], case["D"], 4 if case["weight"] == "fp32" else 2
        if case["op"] == "norm":
            return {"bytes": 2 * T * D * es + 2 * D * ws + 8 * T, "flops": 8 * T * D}
        return {"bytes": 3 * T * D * es + 3 * D * ws + 8 * T, "flops": 14 * T * D}
    T, K, E = case["T"], case["K"], case["E"]
    bytes_ = T * E * es + T * K * case["id_bytes"] + T + 8 * E + 4
    if case["op"] == "balance":
        return {"bytes": bytes_, "flops": 5 * T * E}
    return {"bytes": bytes_ + T * E * es + 4, "flops": 9 * T * E}


# ------------------------------------------------------------------- exact --

def _exact_attend(case, s):
    shards, hq, hkv = _shards(case)
    S, d, queries, window, sinks = case["S"], case["d"], case["queries"], case["window"], case["sinks"]
    ratio, dev = hq // hkv, s["q"].device
    dims = (lambda h, t: (shards, h, t, d)) if case["layout"] == "head" else (lambda h, t: (shards, t, h, d))
    at = (lambda x, n, h: x[n, h]) if case["layout"] == "head" else (lambda x, n, h: x[n, :, h])
    q, k, v = s["q"].view(dims(hq, queries)), s["k"].view(dims(hkv, S)), s["v"].view(dims(hkv, S))
    grad = case["op"] == "attend_grad"
    o = torch.zeros(dims(hq, queries), dtype=torch.float64, device=dev)
    lse = torch.full((shards, hq, queries), -math.inf, dtype=torch.float64, device=dev)
    if grad:
        do = s["do"].view(dims(hq, queries))
        dq, dk, dv = (torch.zeros(dims(h, t), dtype=torch.float64, device=dev) for h, t in ((hq, queries), (hkv, S), (hkv, S)))
    seq = _sequence_of(case, "cpu").tolist()
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    for n in range(shards):
        first, length = starts[seq[n]], lengths[seq[n]]
        lo, hi = max(0, -first), min(queries, length - first)       # the rows that see anything
        for h in range(hq):
            kh, vh = at(k, n, h // ratio), at(v, n, h // ratio)
            for a in range(lo, hi, 4096):
                z = min(hi, a + 4096)
                pos = first + torch.arange(a, z, device=dev)[:, None]
                begin = max(0, first + a - window + 1)
                j = torch.cat([torch.arange(min(sinks, begin), device=dev), torch.arange(begin, first + z, device=dev)])
                off = (j > pos) | ((pos - j >= window) & (j >= sinks))
                kj, vj, qi = kh[j].double(), vh[j].double(), at(q, n, h)[a:z].double()
                sc = (qi @ kj.T * s["scale"]).masked_fill_(off, -math.inf)
                total = torch.logsumexp(sc, 1, keepdim=True)
                p = torch.exp(sc - total)
                oi = p @ vj
                at(o, n, h)[a:z] = oi
                lse[n, h, a:z] = total[:, 0]
                if grad:
                    g = at(do, n, h)[a:z].double()
                    ds = p * (g @ vj.T - (g * oi).sum(1, keepdim=True)) * s["scale"]
                    at(dq, n, h)[a:z] = ds @ kj
                    at(dk, n, h // ratio).index_add_(0, j, ds.T @ qi)
                    at(dv, n, h // ratio).index_add_(0, j, p.T @ g)
    if case["op"] == "attend_step":
        return o.view(-1)
    if not grad:
        return o.view(-1), lse.view(-1)
    return o.view(-1), lse.view(-1), dq.view(-1), dk.view(-1), dv.view(-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("attend"):
        return _exact_attend(case, s)
    if case["op"] == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        return torch.addcmul(s["bias"].double(), (x - mean[:, None]) * s["weight"].double(), rstd[:, None]), mean, rstd
    if case["op"] == "norm_grad":
        # by the derivative of each part of the definition, with the given statistics
        T, D = case["T"], case["D"]
        dy, rstd = s["dy"].double(), s["rstd"].double()
        centred = s["x"].double() - s["mean"].double()[:, None]
        dn = dy * s["weight"].double()
        along = torch.einsum("td,td->t", dn, centred) * rstd ** 3 / D
        dc = dn * rstd[:, None] - centred * along[:, None]
        dx = dc - (rstd * dn.sum(1) / D)[:, None]
        return dx, torch.einsum("td,td,t->d", dy, centred, rstd), torch.ones(T, dtype=torch.float64, device=dy.device) @ dy
    T, K, E = case["T"], case["K"], case["E"]
    rows = torch.nonzero(s["mask"])[:, 0]
    counts = torch.bincount(s["ids"][rows].reshape(-1).long(), minlength=E)
    x = s["logits"][rows].double()
    p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    L = rows.numel()
    share = counts.double() / (L * K)
    loss = COEF * E * torch.dot(share, p.mean(0))
    slope = COEF * E * share / L
    if case["op"] == "balance":
        return loss.view(1), counts.int(), slope
    dlogits = torch.zeros(T, E, dtype=torch.float64, device=x.device)
    dlogits[rows] = s["dloss"].double() * (p * slope - p * (p @ slope)[:, None])
    return loss.view(1), counts.int(), slope, dlogits
