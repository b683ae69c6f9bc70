"""The index-driven re-layouts as they are measured: tokens sorted by expert and
back, and the embedding lookup with its gradient.

``run`` computes each operator in plain torch operations (``own`` false) or
through the library's entry points (``own`` true), on what ``prepare`` made.
``exact`` computes the same from the definitions in 64 bits.

Definitions.  T tokens choose K of E experts each; slot s = t*K + k.  A slot
whose id is outside [0, E) is dropped.  The rows of one expert are the kept
slots with its id in slot order; an expert's rows start at a multiple of
``align``.  ``pos`` is a slot's row (-1: dropped), ``order`` a row's slot (-1:
none), ``offsets`` the experts' first rows and the end, ``counts`` the kept
slots of each expert.

  seq_to_expert       rows[r] = x[order[r] // K], 0 where the row has no slot
  seq_to_expert_grad  dx[t] = sum over k of drows[pos[t, k]]
  expert_to_seq       y[t] = sum over k of w[t, k] * rows[pos[t, k]]
  expert_to_seq_grad  drows[pos[t, k]] = w[t, k] * dy[t], 0 in rows without a
                      slot; dw[t, k] = <dy[t], rows[pos[t, k]]>, 0 if dropped
  embed               y[row(t)] = scale * table[id[t]], 0 where id is outside [0, V)
  embed_grad          dtable[v] = scale * sum over t with id[t] = v of dy[row(t)]

row(t) is the place of token t in the sequence-sharded layout: rank shards in
rank order, each [sequences of the group][tokens of the member].
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IDS = {4: torch.int32, 8: torch.int64}


def listed():
    return [
        # one step of a small serving batch: routing 16 tokens, where the latency of the call counts
        dict(name="route_decode", op="route", T=16, K=4, E=64, D=2048, align=1, dtype="bf16", id_bytes=8, drop=0.0),
        # one micro-batch of two 16k sequences at width 2048, rows padded for experts' products in tiles of 128
        dict(name="route_train", op="route", T=32768, K=4, E=64, D=2048, align=128, dtype="bf16", id_bytes=8, drop=0.0),
        # a ragged fp16 batch with dropped choices: the gradient of the sort
        dict(name="route_grad_ragged", op="route_grad", T=4099, K=3, E=20, D=1000, align=1, dtype="fp16", id_bytes=4,
             drop=0.1),
        # the same gradient for a micro-batch of two 16k sequences at width 4096, two choices a token
        dict(name="route_grad_train", op="route_grad", T=32768, K=2, E=8, D=4096, align=1, dtype="bf16", id_bytes=8,
             drop=0.0),
        # back from the experts for a small serving batch with many choices a token
        dict(name="combine_decode", op="combine", T=16, K=8, E=128, D=4096, align=1, dtype="bf16", id_bytes=8, drop=0.0),
        # back from the experts in training
        dict(name="combine_train", op="combine", T=32768, K=4, E=64, D=2048, align=128, dtype="bf16", id_bytes=8,
             drop=0.0),
        # an odd fp32 width, as a parity run in full precision has it
        dict(name="combine_grad_odd", op="combine_grad", T=1023, K=5, E=40, D=777, align=4, dtype="fp32", id_bytes=4,
             drop=0.2),
        # the largest: eight choices a token, both gradients
        dict(name="combine_grad_train", op="combine_grad", T=16384, K=8, E=128, D=2048, align=1, dtype="bf16", id_bytes=8,
             drop=0.0),
        # the embedding of a small serving batch
        dict(name="embed_decode", op="embed", N=1, B=16, S=1, groups=1, V=131072, D=2048, dtype="bf16", id_bytes=8),
        # two 16k sequences over eight ranks in one group: the rows are re-laid on the way
        dict(name="embed_train", op="embed", N=8, B=2, S=16384, groups=1, V=131072, D=2048, dtype="bf16", id_bytes=8),
        # a small vocabulary in fp32 with an odd width
        dict(name="embed_grad_odd", op="embed_grad", N=1, B=3, S=1365, groups=1, V=8191, D=501, dtype="fp32", id_bytes=4),
        # the gradient of a whole table from two 16k sequences over eight ranks in two groups
        dict(name="embed_grad_train", op="embed_grad", N=8, B=2, S=16384, groups=2, V=131072, D=2048, dtype="bf16",
             id_bytes=8),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "combine", "combine_grad", "embed", "embed_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    id_bytes = rng.choice([4, 8])
    D = _log(rng, 64, 8192)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)
    while True:
        if op.startswith("embed"):
            groups = rng.choice([1, 1, 2, 4])
            members = rng.choice([1, 2, 4])
            case = dict(op=op, N=groups * members, B=groups * rng.choice([1, 2, 3]), S=members * _log(rng, 1, 8192),
                        groups=groups, V=_log(rng, 500, 150000), D=D, dtype=dtype, id_bytes=id_bytes)
        else:
            E = _log(rng, 4, 512)
            case = dict(op=op, T=_log(rng, 1, 32768), K=rng.randint(1, min(8, E)), E=E, D=D,
                        align=rng.choice([1, 1, 8, 16, 128]), dtype=dtype, id_bytes=id_bytes,
                        drop=rng.choice([0.0, 0.0, 0.1, 0.5]))
        if work(case)["bytes"] <= 1.0e9:
            return case


def _max_rows(case):
    M, a = case["T"] * case["K"], case["align"]
    return (M + min(case["E"], M) * (a - 1)) // a * a


def _sequence_sharded(case, per_token):
    """Values given per token in the order [B][S], in the order of the sequence-sharded layout."""
    G = case["groups"]
    P, Bl = case["N"] // G, case["B"] // G
    return per_token.reshape(G, Bl, P, case["S"] // P).transpose(1, 2).reshape(-1)


def _sorted(case, ids):
    """pos, order, offsets and counts of the slots, by a stable sort of their experts."""
    E, a, rows = case["E"], case["align"], _max_rows(case)
    ids = ids.reshape(-1).long()
    M, dev = ids.numel(), ids.device
    key = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=dev).scatter_add_(0, key, torch.ones_like(key))
    counts[E] = 0
    dense = counts.cumsum(0) - counts                      # the last is the number of kept slots
    padded = (counts + a - 1) // a * a
    starts = padded.cumsum(0) - padded
    key_s, slot_s = torch.sort(key, stable=True)
    row_s = torch.arange(M, device=dev) - dense[key_s] + starts[key_s]
    kept = key_s < E
    pos = torch.empty_like(slot_s)
    pos[slot_s] = torch.where(kept, row_s, torch.full_like(row_s, -1))
    order = torch.full((rows + 1,), -1, dtype=torch.int64, device=dev)
    order[torch.where(kept, row_s, torch.full_like(row_s, rows))] = slot_s
    return pos.int(), order[:rows].int(), starts.int(), counts[:E].int()


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(dt)

    if case["op"].startswith("embed"):
        T, V, D = case["B"] * case["S"], case["V"], case["D"]
        # few rows are asked for often and most seldom, as words are
        u = torch.rand(T, generator=g, device=dev, dtype=torch.float64)
        ids = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1).to(IDS[case["id_bytes"]])
        state = dict(case=case, ids=ids, scale=math.sqrt(D))
        if case["op"] == "embed":
            state["table"] = normal(V, D) * 0.02
            state["out"] = torch.empty(T, D, dtype=dt, device=dev)
        else:
            state["dy"] = normal(T, D)
            state["out"] = torch.empty(V, D, dtype=dt, device=dev)
    else:
        T, K, E, D = case["T"], case["K"], case["E"], case["D"]
        rows = _max_rows(case)
        # a router's choices: the largest of noisy scores, some experts liked more than others
        liked = torch.randn(E, generator=g, device=dev)
        scores, ids = torch.topk(torch.randn(T, E, generator=g, device=dev) + 0.5 * liked, K, dim=1)
        weights = torch.softmax(scores, dim=1).contiguous()
        gone = torch.rand(T, K, generator=g, device=dev) < case["drop"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids).to(IDS[case["id_bytes"]]).contiguous()
        i32 = dict(dtype=torch.int32, device=dev)
        state = dict(case=case, ids=ids)
        if case["op"] == "route":
            state.update(x=normal(T, D), pos=torch.empty(T * K, **i32), order=torch.empty(rows, **i32),
                         offsets=torch.empty(E + 1, **i32), counts=torch.empty(E, **i32),
                         rows=torch.empty(rows, D, dtype=dt, device=dev))
        else:
            pos, order, _, _ = _sorted(case, ids)
            state.update(pos=pos, order=order, weights=weights)
        if case["op"] == "route_grad":
            state.update(drows=normal(rows, D), dx=torch.empty(T, D, dtype=dt, device=dev))
        if case["op"] == "combine":
            state.update(rows=normal(rows, D), y=torch.empty(T, D, dtype=dt, device=dev))
        if case["op"] == "combine_grad":
            state.update(rows=normal(rows, D), dy=normal(T, D), drows=torch.empty(rows, D, dtype=dt, device=dev),
                         dw=torch.empty(T, K, device=dev))
    if own:
        state.update(_plan(case))
    return state


def _plan(case):
    """The plan and the workspace that a program keeps for its sizes."""
    from sequence_re_layout_amd import binding as b
    dt = {"bf16": b.BASP_BF16, "fp16": b.BASP_FP16, "fp32": b.BASP_FP32}[case["dtype"]]
    if case["op"].startswith("embed"):
        layout = b.basp_plan_create_groups(case["N"], case["B"], case["S"], case["N"], case["N"], 1, dt, case["groups"])
        plan = b.basp_embed_plan_create(layout, case["B"] * case["S"], case["V"], case["D"], id_bytes=case["id_bytes"],
                                        dtype=dt, grad_dtype=dt)
    else:
        plan = b.basp_expert_plan_create(case["T"], case["K"], case["E"], case["D"], align=case["align"],
                                         id_bytes=case["id_bytes"], dtype=dt, weight_dtype=b.BASP_FP32)
    ws = torch.empty(max(1, plan.info["workspace_bytes"]), dtype=torch.uint8, device="cuda")
    return dict(b=b, plan=plan, ws=ws)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        b, plan = s["b"], s["plan"]
        if op == "route":
            b.basp_route_to_expert(plan, s["x"], s["ids"], s["pos"], s["order"], s["offsets"], s["counts"], s["rows"],
                                   s["ws"])
            return s["pos"], s["order"], s["offsets"], s["counts"], s["rows"]
        if op == "route_grad":
            b.basp_seq_to_expert_grad(plan, s["drows"], s["pos"], s["dx"])
            return s["dx"]
        if op == "combine":
            b.basp_expert_to_seq(plan, s["rows"], s["pos"], s["weights"], s["y"])
            return s["y"]
        if op == "combine_grad":
            b.basp_expert_to_seq_grad(plan, s["dy"], s["rows"], s["pos"], s["order"], s["weights"], s["drows"], s["dw"])
            return s["drows"], s["dw"]
        if op == "embed":
            b.basp_embed_to_seq(plan, s["ids"], s["table"], s["scale"], s["out"])
            return s["out"]
        b.basp_embed_to_seq_grad(plan, s["ids"], s["dy"], s["scale"], False, s["out"], s["ws"])
        return s["out"]
    return _PLAIN[op](s["case"], s)


def _plain_route(case, s):
    pos, order, offsets, counts = _sorted(case, s["ids"])
    token = order.clamp(min=0).long() // case["K"]
    rows = torch.where((order >= 0)[:, None], s["x"][token], torch.zeros((), dtype=s["x"].dtype, device=order.device))
    return pos, order, offsets, counts, rows


def _of_slots(case, rows, pos):
    """The rows of each token's slots in 32 bits, [T][K][D], 0 for dropped slots."""
    g = rows[pos.clamp(min=0).long()].float()
    return g.masked_fill_((pos < 0)[:, None], 0.0).view(case["T"], case["K"], case["D"])


def _plain_route_grad(case, s):
    return _of_slots(case, s["drows"], s["pos"]).sum(1).to(s["drows"].dtype)


def _plain_combine(case, s):
    w = s["weights"].masked_fill(s["pos"].view(case["T"], case["K"]) < 0, 0.0)
    return (_of_slots(case, s["rows"], s["pos"]) * w[:, :, None]).sum(1).to(s["rows"].dtype)


def _plain_combine_grad(case, s):
    dy = s["dy"].float()
    dw = (_of_slots(case, s["rows"], s["pos"]) * dy[:, None, :]).sum(2)
    slot = s["order"].clamp(min=0).long()
    drows = s["weights"].view(-1)[slot][:, None] * dy[slot // case["K"]]
    return drows.masked_fill_((s["order"] < 0)[:, None], 0.0).to(s["dy"].dtype), dw


def _plain_embed(case, s):
    ids = _sequence_sharded(case, s["ids"].long())
    return (s["table"][ids].float() * s["scale"]).to(s["table"].dtype)


def _plain_embed_grad(case, s):
    ids = _sequence_sharded(case, s["ids"].long())
    total = torch.zeros(case["V"], case["D"], device=ids.device).index_add_(0, ids, s["dy"].float())
    return (total * s["scale"]).to(s["dy"].dtype)


_PLAIN = {"route": _plain_route, "route_grad": _plain_route_grad, "combine": _plain_combine,
          "combine_grad": _plain_combine_grad, "embed": _plain_embed, "embed_grad": _plain_embed_grad}


def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    D = case["D"]
    if case["op"].startswith("embed"):
        T, V = case["B"] * case["S"], case["V"]
        # rows asked for twice are read once: the expected number of different ids
        v = np.arange(V, dtype=np.float64)
        used = int((1.0 - (1.0 - np.log1p(1.0 / (v + 1.0)) / math.log(V + 1)) ** T).sum())
        if case["op"] == "embed":
            return {"bytes": T * case["id_bytes"] + (used + T) * D * es, "flops": T * D}
        return {"bytes": T * case["id_bytes"] + (T + V) * D * es, "flops": (T + used) * D}
    T, K, E, rows = case["T"], case["K"], case["E"], _max_rows(case)
    M = T * K
    used = int(M * (1.0 - case["drop"]))
    if case["op"] == "route":
        return {"bytes": M * (case["id_bytes"] + 4) + rows * 4 + (2 * E + 1) * 4 + (T + rows) * D * es, "flops": M}
    if case["op"] == "route_grad":
        return {"bytes": M * 4 + (used + T) * D * es, "flops": used * D}
    if case["op"] == "combine":
        return {"bytes": M * 8 + (used + T) * D * es, "flops": 2 * used * D}
    return {"bytes": M * 12 + rows * 4 + (used + T + rows) * D * es, "flops": 3 * used * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("embed"):
        # the place of every token, rank by rank: member j of group n holds tokens [j*St, (j+1)*St) of its sequences
        B, S, P = case["B"], case["S"], case["N"] // case["groups"]
        Bl, St = B // case["groups"], S // P
        t = torch.arange(B * S, device=s["ids"].device)
        seq, at = t // S, t % S
        place = ((seq // Bl * P + at // St) * Bl + seq % Bl) * St + at % St
        ids = s["ids"].long()
        if case["op"] == "embed":
            out = torch.empty(B * S, case["D"], dtype=torch.float64, device=t.device)
            out[place] = s["table"].double()[ids] * s["scale"]
            return out
        # sums of neighbours in sorted order, as differences of running sums
        ids, by = torch.sort(ids)
        edge = torch.searchsorted(ids, torch.arange(case["V"] + 1, device=t.device))
        total = torch.empty(case["V"], case["D"], dtype=torch.float64, device=t.device)
        for c in range(0, case["D"], 256):
            part = s["dy"][:, c:c + 256].double()[place[by]].cumsum(0)
            part = torch.cat([torch.zeros_like(part[:1]), part])
            total[:, c:c + 256] = part[edge[1:]] - part[edge[:-1]]
        return total * s["scale"]
    T, K, E, a, rows = case["T"], case["K"], case["E"], case["align"], _max_rows(case)
    if case["op"] == "route":
        # each slot's place among the slots of its expert, counted over all slots before it
        of = s["ids"].reshape(-1, 1) == torch.arange(E, device=s["ids"].device)
        before = of.int().cumsum(0, dtype=torch.int32)
        counts = before[-1]
        ends = ((counts + a - 1) // a * a).cumsum(0)
        offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
        pos = ((before - 1 + offsets[:-1]) * of).sum(1).masked_fill(~of.any(1), -1)
        out = torch.zeros(rows, case["D"], dtype=torch.float64, device=pos.device)
        order = torch.full((rows,), -1, dtype=torch.int64, device=pos.device)
        kept = torch.nonzero(pos >= 0)[:, 0]
        order[pos[kept]] = kept
        for c in range(0, case["D"], 256):
            out[pos[kept], c:c + 256] = s["x"][:, c:c + 256].double()[kept // K]
        return pos.int(), order.int(), offsets.int(), counts.int(), out
    pos = s["pos"].view(T, K).long()
    w = s["weights"].double() if case["op"] != "route_grad" else torch.ones(T, K, dtype=torch.float64, device=pos.device)
    if case["op"] == "combine_grad":
        drows = torch.zeros(rows, case["D"], dtype=torch.float64, device=pos.device)
        dw = torch.zeros(T, K, dtype=torch.float64, device=pos.device)
        dy = s["dy"].double()
        for k in range(K):
            t = torch.nonzero(pos[:, k] >= 0)[:, 0]
            p = pos[t, k]
            dw[t, k] = (s["rows"][p].double() * dy[t]).sum(1)
            drows[p] = dy[t] * w[t, k, None]
        return drows, dw
    rows_in = s["drows"] if case["op"] == "route_grad" else s["rows"]
    y = torch.zeros(T, case["D"], dtype=torch.float64, device=pos.device)
    for k in range(K):
        t = torch.nonzero(pos[:, k] >= 0)[:, 0]
        y[t] += w[t, k, None] * rows_in[pos[t, k]].double()
    return y
