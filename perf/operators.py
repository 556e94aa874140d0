"""The gated linear recurrence and the state pool's row operators: the calls
that are measured, their plain forms and their definitions in 64 bits.

``run`` makes one pass: with ``own`` through the package's entry points, else
as elementary torch operations in fp32, rounded once at the end.  ``exact``
follows each definition token by token in fp64.

Operators (``op`` of a case):
  forward   h_t = g_t * h_{t-1} + x_t over packed sequences, with start and
            final states
  training  the same and its gradients
  decode    one token for every sequence, states in pool rows
  copy      pool rows copied (forked) inside a pool or from another one
  reset     pool rows zeroed
  compact   the live rows of a pool moved to its front, indices renamed
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
LARGEST = 65536 * 32 * 128  # elements of the largest listed forward pass


def listed():
    return [
        # a small ragged prefill batch with an empty and a one-token sequence,
        # states in a pool: launch latency
        {"name": "forward ragged 6", "op": "forward", "lens": "130,20,300,0,64,1", "heads": 16,
         "dim": 128, "dtype": "f32", "gate": "f32", "per_head": False, "pool": 64},
        # one long prompt through a wide layer: bandwidth and the long chain
        {"name": "forward long", "op": "forward", "lens": "65536", "heads": 32, "dim": 128,
         "dtype": "bf16", "gate": "f32", "per_head": False, "pool": 0},
        # a training step on two sequences
        {"name": "training 2 x 2048", "op": "training", "lens": "2048,2048", "heads": 16,
         "dim": 128, "dtype": "bf16", "gate": "f32", "per_head": False},
        # a training step on a packed batch of uneven lengths, one gate a head
        # (its gradient is summed over the head's channels)
        {"name": "training packed 8", "op": "training",
         "lens": "8192,1531,2999,61,4097,1,3412,2767", "heads": 32, "dim": 128, "dtype": "f16",
         "gate": "f32", "per_head": True},
        # a few streams, one token each: latency
        {"name": "decode 6", "op": "decode", "seqs": 6, "heads": 16, "dim": 128, "dtype": "f16",
         "gate": "f16", "per_head": False, "state": "f32", "pool": 64},
        # a full serving batch
        {"name": "decode 256", "op": "decode", "seqs": 256, "heads": 32, "dim": 128,
         "dtype": "bf16", "gate": "f32", "per_head": False, "state": "f32", "pool": 512},
        # four prompts forked into eight samples each, fp32 gated-delta states
        {"name": "copy fork 4 x 8", "op": "copy", "rows": 64, "row": "16,128,128", "from": "f32",
         "to": "f32", "sources": 4, "copies": 32, "same": True},
        # bf16 checkpoints brought back into an fp32 pool
        {"name": "copy checkpoints", "op": "copy", "rows": 128, "row": "32,128,128",
         "from": "bf16", "to": "f32", "sources": 96, "copies": 96, "same": False},
        # rows of a recurrence pool taken for new sequences: latency
        {"name": "reset 8 small", "op": "reset", "rows": 512, "row": "16,128", "to": "f32",
         "copies": 8},
        # gated-delta rows taken for a new batch
        {"name": "reset 64", "op": "reset", "rows": 128, "row": "16,128,128", "to": "f32",
         "copies": 64},
        # a recurrence pool after half of its sequences ended
        {"name": "compact 512 small", "op": "compact", "rows": 512, "row": "16,128", "to": "f32",
         "live": 256},
        # a gated-delta pool after half of its sequences ended
        {"name": "compact 256", "op": "compact", "rows": 256, "row": "16,128,128", "to": "bf16",
         "live": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _layer(rng):
    per_head = rng.random() < 0.4
    if per_head:
        dim = rng.choice([32, 64, 128])
    else:
        dim = rng.choice([32, 64, 128, 128, 128, _log_int(rng, 1, 256)])
    dtype = rng.choice(["f32", "bf16", "f16"])
    return {"heads": _log_int(rng, 1, 32), "dim": dim, "dtype": dtype,
            "gate": rng.choice(["f32", dtype]), "per_head": per_head}


def _lens(rng, most_tokens):
    total = _log_int(rng, 1, max(1, most_tokens))
    n = _log_int(rng, 1, 256)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["forward", "training", "decode", "copy", "reset", "compact"])
    if op in ("forward", "training"):
        case = dict(_layer(rng), op=op)
        # a training pass moves about three times a forward pass's bytes
        most = LARGEST // (4 if op == "training" else 2) // (case["heads"] * case["dim"])
        case["lens"] = _lens(rng, min(131072, most))
        if op == "forward":
            n = case["lens"].count(",") + 1
            case["pool"] = rng.choice([0, n + rng.randint(0, 64)])
        return case
    if op == "decode":
        n = _log_int(rng, 1, 1024)
        return dict(_layer(rng), op=op, seqs=n, pool=n + rng.randint(0, n),
                    state=rng.choice(["f32", "bf16", "f16"]))
    if rng.random() < 0.5:  # a recurrence pool, else a gated-delta pool
        row, most = "%d,%d" % (_log_int(rng, 1, 32), rng.choice([32, 64, 128, _log_int(rng, 1, 256)])), 1024
    else:
        dim = rng.choice([32, 64, 128])
        row, most = "%d,%d,%d" % (_log_int(rng, 1, 32), dim, dim), 128
    rows = _log_int(rng, 8, most)
    to = rng.choice(["f32", "bf16", "f16"])
    if op == "compact":
        return {"op": op, "rows": rows, "row": row, "to": to, "live": rng.randint(1, rows)}
    if op == "reset":
        return {"op": op, "rows": rows, "row": row, "to": to, "copies": rng.randint(1, rows)}
    same = rng.random() < 0.5
    copies = rng.randint(1, max(1, rows // 2))
    return {"op": op, "rows": rows, "row": row, "from": to if same else rng.choice(list(DTYPES)),
            "to": to, "sources": rng.randint(1, copies), "copies": copies, "same": same}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _gates(case, tokens, gen):
    """Forget gates exp(-rate * softplus(z)): rates spread over three decades,
    so that some channels (or heads) forget in a token and some in thousands."""
    shape = (case["heads"],) if case["per_head"] else (case["heads"], case["dim"])
    rate = torch.exp(math.log(1e-3) * torch.rand(shape, generator=gen, device="cuda"))
    z = torch.randn((tokens,) + shape, generator=gen, device="cuda")
    return torch.exp_(torch.nn.functional.softplus(z).mul_(-rate)).to(DTYPES[case["gate"]])


def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def some_rows(most, n):
        return torch.randperm(most, generator=gen, device="cuda")[:n]

    s = {"case": case}
    if op in ("forward", "training"):
        lens = _ints(case["lens"])
        n, tokens, hd = len(lens), sum(lens), (case["heads"], case["dim"])
        s["lens"] = lens
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["x"] = _normal((tokens,) + hd, case["dtype"], gen)
        s["g"] = _gates(case, tokens, gen)
        if op == "training":
            s["h0"] = _normal((n,) + hd, "f32", gen)
            s["dout"] = _normal((tokens,) + hd, case["dtype"], gen)
            s["dfinal"] = _normal((n,) + hd, "f32", gen)
        elif case["pool"]:
            s["h0"] = _normal((case["pool"],) + hd, "f32", gen)
            s["final"] = torch.zeros_like(s["h0"])
            s["idx"] = some_rows(case["pool"], n).to(torch.int32)
        else:
            s["h0"] = _normal((n,) + hd, "f32", gen)
        return s
    if op == "decode":
        n, hd = case["seqs"], (case["heads"], case["dim"])
        s["x"] = _normal((n,) + hd, case["dtype"], gen)
        s["g"] = _gates(case, n, gen)
        s["h0"] = _normal((case["pool"],) + hd, case["state"], gen)
        s["final"] = torch.zeros_like(s["h0"])
        s["idx"] = some_rows(case["pool"], n).to(torch.int32)
        return s
    row = tuple(_ints(case["row"]))
    s["pool"] = _normal((case["rows"],) + row, case["to"], gen)
    if op == "copy":
        if case["same"]:  # sources and destinations apart
            at = some_rows(case["rows"], case["sources"] + case["copies"])
            src, s["dst"] = at[:case["sources"]], at[case["sources"]:].to(torch.int32)
        else:
            s["from"] = _normal((case["sources"],) + row, case["from"], gen)
            src = some_rows(case["sources"], case["sources"])
            s["dst"] = some_rows(case["rows"], case["copies"]).to(torch.int32)
        s["src"] = src[torch.arange(s["dst"].numel(), device="cuda") % src.numel()].to(torch.int32)
    elif op == "reset":
        s["at"] = some_rows(case["rows"], case["copies"]).to(torch.int32)
    else:
        s["idx"] = some_rows(case["rows"], case["live"]).to(torch.int32)
    return s


# --------------------------------------------------------------- plain forms

def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling the span that
    each element covers; a is 0 where a sequence starts."""
    span = 1
    while span < longest:
        b = torch.cat([b[:span], torch.addcmul(b[span:], a[span:], b[:-span])])
        if 2 * span < longest:
            a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _bounds(s):
    """First and last tokens of the sequences that have any, and their numbers."""
    ends = torch.tensor(s["lens"]).cumsum(0)
    some = torch.tensor([i for i, n in enumerate(s["lens"]) if n], dtype=torch.long)
    first = ends[some] - torch.tensor(s["lens"])[some]
    return [t.to("cuda", non_blocking=True) for t in (first, ends[some] - 1, some)]


def _wide(g):
    return g.float() if g.dim() == 3 else g.float().unsqueeze(-1)


def _plain_forward(s, h0):
    first, last, some = _bounds(s)
    x, g = s["x"].float(), _wide(s["g"])
    b = x.index_add(0, first, (g[first] * h0[some]))
    a = g.index_fill(0, first, 0.0).expand_as(x).contiguous()
    h = _scan(a, b, max(s["lens"]))
    return h, h0.index_copy(0, some, h[last])


def _plain_training(s):
    first, last, some = _bounds(s)
    h, final = _plain_forward(s, s["h0"])
    g = _wide(s["g"])
    d = s["dout"].float().index_add(0, last, s["dfinal"][some])
    a = torch.cat([g[1:], g[:1]]).index_fill(0, last, 0.0).expand_as(d)
    dh = _scan(a.flip(0), d.flip(0), max(s["lens"])).flip(0)
    before = torch.cat([h[:1], h[:-1]]).index_copy(0, first, s["h0"][some])
    dg = dh * before
    dg = dg.sum(-1) if s["case"]["per_head"] else dg
    dh0 = s["dfinal"].index_copy(0, some, g[first] * dh[first])
    return (h.to(s["x"].dtype), final, dh.to(s["x"].dtype), dg.to(s["g"].dtype), dh0)


def _plain_compact(pool, idx):
    rows = torch.arange(pool.shape[0], device=pool.device)
    live = torch.zeros(pool.shape[0], dtype=torch.bool, device=pool.device)
    live[idx.long()] = True
    m = live.sum()
    hole, mover = ~live & (rows < m), live & (rows >= m)
    where = rows.clone()
    moved = mover.nonzero()[:, 0]
    where[moved] = hole.nonzero()[:, 0]
    pool[where[moved]] = pool[moved]
    return pool, where[idx.long()].to(idx.dtype), m.to(torch.int32).reshape(1)


def _plain(s):
    op = s["case"]["op"]
    if op == "forward":
        if "idx" not in s:
            h, final = _plain_forward(s, s["h0"])
            return h.to(s["x"].dtype), final
        idx = s["idx"].long()
        h, final = _plain_forward(s, s["h0"][idx])
        s["final"][idx] = final
        return h.to(s["x"].dtype), s["final"]
    if op == "training":
        return _plain_training(s)
    if op == "decode":
        idx = s["idx"].long()
        h = torch.addcmul(s["x"].float(), _wide(s["g"]), s["h0"][idx].float())
        s["final"][idx] = h.to(s["final"].dtype)
        return h.to(s["x"].dtype), s["final"]
    pool = s["pool"]
    if op == "copy":
        pool[s["dst"].long()] = s.get("from", pool)[s["src"].long()].to(pool.dtype)
        return pool
    if op == "reset":
        pool[s["at"].long()] = 0
        return pool
    return _plain_compact(pool, s["idx"])


def _own(s):
    import gated_deltanet_chunked_varlen_amd as gdn
    op = s["case"]["op"]
    if op == "forward":
        if "idx" not in s:
            return gdn.gated_linear_recurrence(s["x"], s["g"], initial_state=s["h0"],
                                               output_final_state=True, cu_seqlens=s["cu"])
        return gdn.gated_linear_recurrence(s["x"], s["g"], initial_state=s["h0"],
                                           output_final_state=True, cu_seqlens=s["cu"],
                                           output_state=s["final"], state_indices=s["idx"])
    if op == "training":
        out, final, kept = gdn.gated_linear_recurrence(
            s["x"], s["g"], initial_state=s["h0"], output_final_state=True,
            cu_seqlens=s["cu"], return_chunk_states=True)
        dx, dg, dh0 = gdn.gated_linear_recurrence_backward(
            s["dout"], s["x"], s["g"], initial_state=s["h0"], dfinal_state=s["dfinal"],
            cu_seqlens=s["cu"], chunk_states=kept, output_dinitial_state=True)
        return out, final, dx, dg, dh0
    if op == "decode":
        return gdn.gated_linear_recurrence_decode(s["x"], s["g"], initial_state=s["h0"],
                                                  output_state=s["final"], state_indices=s["idx"])
    if op == "copy":
        return gdn.state_pool_copy(s["pool"], s["src"], s["dst"], src_pool=s.get("from"))
    if op == "reset":
        return gdn.state_pool_reset(s["pool"], s["at"])
    idx, live = gdn.state_pool_compact(s["pool"], s["idx"])
    return s["pool"], idx, live


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op in ("forward", "training", "decode"):
        lens = _ints(case["lens"]) if "lens" in case else [1] * case["seqs"]
        n, tokens, row = len(lens), sum(lens), case["heads"] * case["dim"]
        e, es = tokens * row, SIZES[case["dtype"]]
        gate = tokens * (case["heads"] if case["per_head"] else row) * SIZES[case["gate"]]
        if op == "decode":
            return {"bytes": 2 * e * es + gate + 2 * n * row * SIZES[case["state"]], "flops": 2 * e}
        if op == "forward":
            return {"bytes": 2 * e * es + gate + 8 * n * row, "flops": 2 * e}
        # forward: x, g, h0 -> out, final; backward: x, g, dout, h0, dfinal -> dx, dg, dh0
        return {"bytes": 5 * e * es + 3 * gate + 20 * n * row, "flops": 8 * e}
    row = math.prod(_ints(case["row"]))
    if op == "copy":
        read = case["sources"] * row * SIZES[case["from"]]
        return {"bytes": read + case["copies"] * row * SIZES[case["to"]], "flops": 0}
    if op == "reset":
        return {"bytes": case["copies"] * row * SIZES[case["to"]], "flops": 0}
    # about live * (rows - live) / rows of the live rows lie behind the first `live` ones
    moved = case["live"] * (case["rows"] - case["live"]) // case["rows"]
    return {"bytes": 2 * moved * row * SIZES[case["to"]] + 8 * case["live"], "flops": 0}


# --------------------------------------------------- the definitions, in fp64

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("forward", "training"):
        return _exact_recurrence(s, op == "training")
    if op == "decode":
        out, final = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda"), s["final"].double()
        for i, r in enumerate(s["idx"].tolist()):
            g = s["g"][i].double()
            out[i] = (g if g.dim() == 2 else g[:, None]) * s["h0"][r].double() + s["x"][i].double()
            final[r] = out[i]
        return out, final
    pool = s["pool"].double()
    if op == "copy":
        source = s["from"].double() if "from" in s else pool.clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[b] = source[a]
        return pool
    if op == "reset":
        for r in s["at"].tolist():
            pool[r] = 0
        return pool
    live = sorted(set(s["idx"].tolist()))
    holes = [r for r in range(len(live)) if r not in set(live)]
    to = dict(zip([r for r in live if r >= len(live)], holes))
    for a, b in to.items():
        pool[b] = s["pool"][a].double()
    return pool, None, None


def _exact_recurrence(s, training):
    x, g = s["x"].double(), s["g"].double()
    g = g if g.dim() == 3 else g.unsqueeze(-1)
    rows = s["idx"].tolist() if "idx" in s else range(len(s["lens"]))
    final = s["final"].double() if "idx" in s else s["h0"].double().clone()
    out, t, begins = torch.empty_like(x), 0, []
    for r, n in zip(rows, s["lens"]):
        h = s["h0"][r].double()
        begins.append(t)
        for _ in range(n):
            h = torch.addcmul(x[t], g[t], h)
            out[t] = h
            t += 1
        final[r] = h
    if not training:
        return out, final
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    dh0 = torch.empty_like(final)
    for i, (t0, n) in enumerate(zip(begins, s["lens"])):
        back = s["dfinal"][i].double()
        for t in range(t0 + n - 1, t0 - 1, -1):
            d = s["dout"][t].double() + back
            dx[t] = d
            back = g[t] * d
        before = torch.cat([s["h0"][i:i + 1].double(), out[t0:t0 + n - 1]])[:n]
        dg[t0:t0 + n] = dx[t0:t0 + n] * before
        dh0[i] = back
    return out, final, dx, dg.sum(-1) if s["case"]["per_head"] else dg, dh0
