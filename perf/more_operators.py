"""The short causal convolution, the selective state space scan and beam search
over state pools: the calls that are measured, their plain forms and their
definitions in 64 bits.

``run`` makes one pass: with ``own`` through the package's entry points, else
as elementary torch operations in fp32 (beam scores in fp64: they are compared
with each other), rounded once at the end.  ``exact`` follows each definition
token by token, or by a full sort, in fp64.

Operators (``op`` of a case):
  conv           short causal convolution of packed sequences, states in rows
  conv training  the same and its gradients
  conv decode    one token for every sequence
  scan           selective state space scan of packed sequences
  scan training  the same and its gradients
  scan decode    one token for every sequence
  select         the best continuations of the beams of each group
  reorder        pool rows brought in the order of the selected parents
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
LARGEST_CONV = 23060 * 8192     # tokens x channels of the largest listed training pass
LARGEST_SCAN = 16384 * 4096 * 16  # tokens x channels x states of the largest forward pass
LARGEST_LOGITS = 64 * 8 * 131072


def listed():
    return [
        # q, k and v of a small ragged prefill batch with an empty and a
        # one-token sequence, states in a pool: launch latency
        {"name": "conv ragged 6", "op": "conv", "lens": "130,20,300,0,64,1", "channels": 6144,
         "width": 4, "dtype": "bf16", "weight": "bf16", "silu": True, "bias": False, "pool": 64},
        # a training step on a packed batch of uneven lengths, 16 + 16 + 32
        # heads of 128: bandwidth
        {"name": "conv training packed 8", "op": "conv training",
         "lens": "8192,1531,2999,61,4097,1,3412,2767", "channels": 8192, "width": 4,
         "dtype": "bf16", "weight": "f32", "silu": True, "bias": True},
        # a full serving batch
        {"name": "conv decode 256", "op": "conv decode", "seqs": 256, "channels": 8192, "width": 4,
         "dtype": "bf16", "weight": "bf16", "silu": True, "bias": False, "state": "bf16",
         "pool": 512},
        # a small ragged prefill batch, states in a pool: latency of the chain
        {"name": "scan ragged 6", "op": "scan", "lens": "130,20,300,0,64,1", "channels": 2048,
         "states": 16, "groups": 1, "dtype": "f32", "softplus": True, "gated": False, "pool": 64},
        # one long prompt through a wide layer
        {"name": "scan long", "op": "scan", "lens": "16384", "channels": 4096, "states": 16,
         "groups": 1, "dtype": "bf16", "softplus": True, "gated": True, "pool": 0},
        # a training step on two sequences
        {"name": "scan training 2 x 2048", "op": "scan training", "lens": "2048,2048",
         "channels": 4096, "states": 16, "groups": 1, "dtype": "bf16", "softplus": True,
         "gated": True},
        # a few streams, one token each: latency
        {"name": "scan decode 6", "op": "scan decode", "seqs": 6, "channels": 2048, "states": 16,
         "groups": 1, "dtype": "f16", "softplus": True, "gated": True, "state": "f32", "pool": 64},
        # a full serving batch
        {"name": "scan decode 256", "op": "scan decode", "seqs": 256, "channels": 4096,
         "states": 16, "groups": 1, "dtype": "bf16", "softplus": True, "gated": True,
         "state": "f32", "pool": 512},
        # one request of four beams: latency
        {"name": "select 1 x 4", "op": "select", "batch": 1, "beams": 4, "vocab": 32001,
         "candidates": 8, "dtype": "f32"},
        # a full serving batch over a large vocabulary: bandwidth
        {"name": "select 64 x 8", "op": "select", "batch": 64, "beams": 8, "vocab": 131072,
         "candidates": 16, "dtype": "bf16"},
        # short rows of a recurrence pool, two requests of four beams: latency
        {"name": "reorder 2 x 4 small", "op": "reorder", "batch": 2, "beams": 4, "rows": 64,
         "row": "16,128", "to": "f32"},
        # gated-delta rows of a full batch
        {"name": "reorder 16 x 8", "op": "reorder", "batch": 16, "beams": 8, "rows": 128,
         "row": "16,128,128", "to": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(rng, most_tokens):
    total = _log_int(rng, 1, max(1, most_tokens))
    n = _log_int(rng, 1, 256)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def _draw_conv(rng, op):
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    case = {"op": op, "channels": rng.choice([_log_int(rng, 1, 8192), 64 * _log_int(rng, 1, 128)]),
            "width": rng.choice([2, 3, 4, 4]), "dtype": dtype, "weight": rng.choice(["f32", dtype]),
            "silu": rng.random() < 0.7, "bias": rng.random() < 0.5}
    if op == "conv decode":
        n = _log_int(rng, 1, 1024)
        return dict(case, seqs=n, pool=n + rng.randint(0, n), state=rng.choice(["f32", dtype]))
    most = LARGEST_CONV // (4 if dtype == "f32" else 2) // case["channels"]
    case["lens"] = _lens(rng, min(65536, most))
    if op == "conv":
        case["pool"] = rng.choice([0, case["lens"].count(",") + 1 + rng.randint(0, 64)])
    return case


def _draw_scan(rng, op):
    channels = rng.choice([_log_int(rng, 1, 4096), 128 * _log_int(rng, 1, 32)])
    case = {"op": op, "channels": channels,
            "states": rng.choice([16, 16, 16, 8, 64, _log_int(rng, 1, 64)]),
            "groups": rng.choice([g for g in (1, 1, 1, 2, 4, 8) if channels % g == 0]),
            "dtype": rng.choice(["f32", "bf16", "bf16", "f16"]), "softplus": rng.random() < 0.7,
            "gated": rng.random() < 0.6}
    if op == "scan decode":
        n = _log_int(rng, 1, 512)
        return dict(case, seqs=n, pool=n + rng.randint(0, n),
                    state=rng.choice(["f32", "f32", case["dtype"]]))
    # a training pass costs about eight times a forward pass
    most = LARGEST_SCAN // (16 if op == "scan training" else 2) // (channels * case["states"])
    case["lens"] = _lens(rng, min(32768 if op == "scan" else 8192, most))
    if op == "scan":
        case["pool"] = rng.choice([0, case["lens"].count(",") + 1 + rng.randint(0, 64)])
    return case


def draw(rng):
    op = rng.choice(["conv", "conv training", "conv decode", "scan", "scan training",
                     "scan decode", "select", "reorder"])
    if op.startswith("conv"):
        return _draw_conv(rng, op)
    if op.startswith("scan"):
        return _draw_scan(rng, op)
    beams = rng.choice([1, 2, 4, 8, _log_int(rng, 1, 32)])
    batch = _log_int(rng, 1, 64)
    if op == "select":
        vocab = min(_log_int(rng, 1000, 262144), LARGEST_LOGITS // 2 // (batch * beams))
        return {"op": op, "batch": batch, "beams": beams, "vocab": vocab,
                "candidates": beams * rng.randint(1, 2),
                "dtype": rng.choice(["f32", "bf16", "f16"])}
    if rng.random() < 0.5:  # a recurrence or convolution pool, else a gated-delta pool
        row = "%d,%d" % (_log_int(rng, 1, 32), rng.choice([32, 64, 128, _log_int(rng, 1, 256)]))
    else:
        dim = rng.choice([32, 64, 128])
        row = "%d,%d,%d" % (_log_int(rng, 1, 16), dim, dim)
        batch = max(1, min(batch, 128 // beams))
    return {"op": op, "batch": batch, "beams": beams, "rows": batch * beams + rng.randint(0, 16),
            "row": row, "to": rng.choice(["f32", "bf16", "f16"])}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _normal(shape, dtype, gen, by=1.0):
    return (by * torch.randn(shape, generator=gen, device="cuda")).to(DTYPES[dtype])


def _rows(most, n, gen):
    return torch.randperm(most, generator=gen, device="cuda")[:n].to(torch.int32)


def _prepare_sequences(s, case, tokens, n, row, gen):
    """Sequence bounds and states: rows of a pool for serving, one a sequence
    for training."""
    if "seqs" in case:
        s["h0"] = _normal((case["pool"],) + row, case["state"], gen)
        s["final"] = torch.zeros_like(s["h0"])
        s["idx"] = _rows(case["pool"], n, gen)
        return
    s["cu"] = torch.tensor([0] + s["lens"], device="cuda").cumsum(0).to(torch.int32)
    if case["op"].endswith("training"):
        s["h0"] = _normal((n,) + row, "f32", gen)
        s["dout"] = _normal((tokens, case["channels"]), case["dtype"], gen)
        s["dfinal"] = _normal((n,) + row, "f32", gen)
    elif case["pool"]:
        s["h0"] = _normal((case["pool"],) + row, "f32", gen)
        s["final"] = torch.zeros_like(s["h0"])
        s["idx"] = _rows(case["pool"], n, gen)
    else:
        s["h0"] = _normal((n,) + row, "f32", gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op.startswith(("conv", "scan")):
        s["lens"] = _ints(case["lens"]) if "lens" in case else [1] * case["seqs"]
        n, tokens, c, dtype = len(s["lens"]), sum(s["lens"]), case["channels"], case["dtype"]
        s["x"] = _normal((tokens, c), dtype, gen)
    if op.startswith("conv"):
        s["w"] = _normal((c, case["width"]), case["weight"], gen, case["width"] ** -0.5)
        s["bias"] = _normal((c,), case["weight"], gen, 0.1) if case["bias"] else None
        _prepare_sequences(s, case, tokens, n, (case["width"] - 1, c), gen)
    elif op.startswith("scan"):
        ns, g = case["states"], case["groups"]
        # step sizes spread over 0.001 to 0.1, decay rates over 1 to 16
        step = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(c, generator=gen, device="cuda"))
        bias = step + torch.log(-torch.expm1(-step))
        raw = torch.randn((tokens, c), generator=gen, device="cuda")
        if case["softplus"]:
            s["delta"], s["dbias"] = (0.5 * raw).to(DTYPES[dtype]), bias
        else:
            s["delta"], s["dbias"] = (step * torch.exp(0.5 * raw)).to(DTYPES[dtype]), None
        s["A"] = -torch.exp(math.log(16.0) * torch.rand((c, ns), generator=gen, device="cuda"))
        s["B"] = _normal((tokens, g, ns), dtype, gen)
        s["C"] = _normal((tokens, g, ns), dtype, gen)
        s["D"] = _normal((c,), "f32", gen)
        s["z"] = _normal((tokens, c), dtype, gen) if case["gated"] else None
        _prepare_sequences(s, case, tokens, n, (c, ns), gen)
    elif op == "select":
        b, k, v = case["batch"], case["beams"], case["vocab"]
        s["logits"] = _normal((b, k, v), case["dtype"], gen, 3.0)
        # tokens that a constraint forbids, and beams that have ended
        s["logits"][torch.rand((b, k, v), generator=gen, device="cuda") < 0.01] = -math.inf
        s["scores"] = -10.0 * torch.rand((b, k), generator=gen, device="cuda")
        s["scores"][torch.rand((b, k), generator=gen, device="cuda") < 0.05] = -math.inf
    else:
        b, k = case["batch"], case["beams"]
        s["pool"] = _normal((case["rows"],) + tuple(_ints(case["row"])), case["to"], gen)
        s["idx"] = _rows(case["rows"], b * k, gen)
        s["parents"] = torch.randint(k, (b, k), generator=gen, device="cuda").to(torch.int32)
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


def _states(s):
    return s["h0"][s["idx"].long()].float() if "idx" in s else s["h0"].float()


def _with_states(s, out, final):
    if "idx" not in s:
        return out, final
    s["final"][s["idx"].long()] = final.to(s["final"].dtype)
    return out, s["final"]


def _conv_taps(s):
    """Rows that token t's taps and a sequence's final state read, in the
    tokens followed by the initial states."""
    keep = s["case"]["width"] - 1
    lens = torch.tensor(s["lens"])
    tokens, n = int(lens.sum()), len(s["lens"])
    first = lens.cumsum(0) - lens
    seq = torch.repeat_interleave(torch.arange(n), lens)
    back = torch.arange(-keep, 1)

    def rows(at, seq, first):  # token at - first of sequence seq
        pos = at - first
        return torch.where(pos >= 0, at, tokens + seq * keep + keep + pos)

    taps = rows(torch.arange(tokens)[:, None] + back, seq[:, None], first[seq][:, None])
    ends = rows((first + lens)[:, None] + back[:-1], torch.arange(n)[:, None], first[:, None])
    return taps.to("cuda", non_blocking=True), ends.to("cuda", non_blocking=True)


def _plain_conv(s):
    training = s["case"]["op"] == "conv training"
    c, silu = s["case"]["channels"], s["case"]["silu"]
    taps, ends = _conv_taps(s)
    rows = torch.cat([s["x"].float(), _states(s).reshape(-1, c)])
    w = s["w"].float().t()
    window = rows[taps]
    pre = (window * w).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    sig = torch.sigmoid(pre)
    out = (pre * sig if silu else pre).to(s["x"].dtype)
    final = rows[ends]
    if not training:
        return _with_states(s, out, final)
    d = s["dout"].float()
    if silu:
        d = d * (sig * (1 + pre * (1 - sig)))
    drows = torch.zeros_like(rows)
    drows.index_add_(0, taps.reshape(-1), (d[:, None, :] * w).reshape(-1, c))
    drows.index_add_(0, ends.reshape(-1), s["dfinal"].reshape(-1, c))
    dw = (d[:, None, :] * window).sum(0, dtype=torch.float64).t().float()
    tokens = d.shape[0]
    grads = (drows[:tokens].to(s["x"].dtype), dw, drows[tokens:].reshape(s["h0"].shape))
    if s["bias"] is not None:
        grads += (d.sum(0, dtype=torch.float64).float(),)
    return (out, final) + grads


def _plain_scan(s):
    case = s["case"]
    training = case["op"] == "scan training"
    tokens, c, g, ns = s["x"].shape[0], case["channels"], case["groups"], case["states"]
    first, last, some = _bounds(s)
    x, raw = s["x"].float(), s["delta"].float()
    if s["dbias"] is not None:
        raw = raw + s["dbias"]
    dt = torch.logaddexp(raw, torch.zeros_like(raw)) if case["softplus"] else raw
    decay = torch.exp(dt[:, :, None] * s["A"])
    bb = s["B"].float().repeat_interleave(c // g, 1)
    cc = s["C"].float().repeat_interleave(c // g, 1)
    h0 = _states(s)
    h = (dt * x)[:, :, None] * bb
    h.index_add_(0, first, decay[first] * h0[some])
    h = _scan(decay.index_fill(0, first, 0.0), h, max(s["lens"]))
    y = (h * cc).sum(-1) + s["D"] * x
    if case["gated"]:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        out = y * (z * sig)
    else:
        out = y
    out = out.to(s["x"].dtype)
    final = h0.index_copy(0, some, h[last])
    if not training:
        return _with_states(s, out, final)
    d = s["dout"].float()
    dz = ()
    if case["gated"]:
        dz = ((d * y * (sig * (1 + z * (1 - sig)))).to(s["x"].dtype),)
        d = d * (z * sig)
    dh = d[:, :, None] * cc
    dh.index_add_(0, last, s["dfinal"][some])
    follow = torch.cat([decay[1:], decay[:1]]).index_fill(0, last, 0.0)
    dh = _scan(follow.flip(0), dh.flip(0), max(s["lens"])).flip(0)
    dcc = (d[:, :, None] * h).reshape(tokens, g, c // g, ns).sum(2).to(s["x"].dtype)
    before = torch.cat([h[:1], h[:-1]]).index_copy(0, first, h0[some])
    ddecay = dh * before * decay
    dbb = (dh * (dt * x)[:, :, None]).reshape(tokens, g, c // g, ns).sum(2).to(s["x"].dtype)
    du = (dh * bb).sum(-1)
    dA = (ddecay * dt[:, :, None]).sum(0, dtype=torch.float64).float()
    draw_ = (ddecay * s["A"]).sum(-1) + du * x
    if case["softplus"]:
        draw_ = draw_ * torch.sigmoid(raw)
    dh0 = s["dfinal"].index_copy(0, some, decay[first] * dh[first])
    grads = ((du * dt + s["D"] * d).to(s["x"].dtype), draw_.to(s["x"].dtype), dA, dbb, dcc,
             (d * x).sum(0, dtype=torch.float64).float(), dh0) + dz
    if s["dbias"] is not None:
        grads += (draw_.sum(0, dtype=torch.float64).float(),)
    return (out, final) + grads


def _plain_select(s):
    """The best of each beam by whole keys (logit, then lowest token), then the
    best of the group by score, then beam and token."""
    logits, scores, m = s["logits"].float(), s["scores"], s["case"]["candidates"]
    b, k, v = logits.shape
    live = (scores > -math.inf)[:, :, None] & (logits > -math.inf)
    logits = torch.where(live, logits, -math.inf) + 0.0
    bits = logits.view(torch.int32)
    order = bits ^ ((bits >> 31) & 0x7fffffff)  # as the floats are ordered
    key = order.long() * 2 ** 31 + (v - 1 - torch.arange(v, device="cuda"))
    best = torch.topk(key, min(m, v), dim=-1).values
    tokens = v - 1 - (best & (2 ** 31 - 1))
    top = logits.amax(-1, keepdim=True).double()
    top = torch.where(top > -math.inf, top, 0.0)
    total = torch.log(torch.exp(logits.double() - top).sum(-1, keepdim=True))
    value = torch.gather(logits, -1, tokens).double()
    value = torch.where(value > -math.inf, scores.double()[:, :, None] + (value - top - total),
                        -math.inf).reshape(b, -1)
    flat = (torch.arange(k, device="cuda")[:, None] * v + tokens).reshape(b, -1)
    by_place = torch.argsort(flat, dim=-1)
    by_value = torch.argsort(torch.gather(value, -1, by_place), dim=-1, descending=True, stable=True)
    at = torch.gather(by_place, -1, by_value)[:, :m]
    flat = torch.gather(flat, -1, at)
    return (torch.gather(value, -1, at).float(), (flat // v).to(torch.int32),
            (flat % v).to(torch.int32))


def _plain_reorder(s):
    b, k = s["parents"].shape
    parents, idx, pool = s["parents"].long(), s["idx"].reshape(b, k), s["pool"]
    same = parents[:, :, None] == parents[:, None, :]
    more = same.tril(-1).any(-1)  # an earlier child has kept the parent's row
    used = (parents[:, :, None] == torch.arange(k, device="cuda")).any(1)
    source = torch.gather(idx, 1, parents)
    free = idx[~used]
    pool[free.long()] = pool[source[more].long()]
    new = source.masked_scatter(more, free)
    return pool, new.reshape(-1)


def _plain(s):
    op = s["case"]["op"]
    if op.startswith("conv"):
        return _plain_conv(s)
    if op.startswith("scan"):
        return _plain_scan(s)
    return _plain_select(s) if op == "select" else _plain_reorder(s)


def _own(s):
    import gated_deltanet_chunked_varlen_amd as gdn
    case, op = s["case"], s["case"]["op"]
    pooled = {"output_state": s["final"], "state_indices": s["idx"]} if "final" in s else {}
    if op.startswith("conv"):
        layer = {"bias": s["bias"], "activation": "silu" if case["silu"] else None}
        if op == "conv decode":
            return gdn.short_convolution_decode(s["x"], s["w"], initial_state=s["h0"], **layer,
                                                **pooled)
        out, final = gdn.short_convolution(s["x"], s["w"], initial_state=s["h0"],
                                           output_final_state=True, cu_seqlens=s["cu"], **layer,
                                           **pooled)
        if op == "conv":
            return out, final
        dx, dw, db, dh0 = gdn.short_convolution_backward(
            s["dout"], s["x"], s["w"], initial_state=s["h0"], dfinal_state=s["dfinal"],
            cu_seqlens=s["cu"], output_dinitial_state=True, **layer)
        return (out, final, dx, dw, dh0) + (() if db is None else (db,))
    if op.startswith("scan"):
        layer = {"D": s["D"], "z": s["z"], "delta_bias": s["dbias"],
                 "delta_softplus": case["softplus"]}
        args = (s["x"], s["delta"], s["A"], s["B"], s["C"])
        if op == "scan decode":
            return gdn.selective_scan_decode(*args, initial_state=s["h0"], **layer, **pooled)
        if op == "scan":
            return gdn.selective_scan(*args, initial_state=s["h0"], output_final_state=True,
                                      cu_seqlens=s["cu"], **layer, **pooled)
        out, final, kept = gdn.selective_scan(*args, initial_state=s["h0"], output_final_state=True,
                                              cu_seqlens=s["cu"], return_chunk_states=True, **layer)
        dx, ddelta, dA, dB, dC, dD, dz, dbias, dh0 = gdn.selective_scan_backward(
            s["dout"], *args, initial_state=s["h0"], dfinal_state=s["dfinal"], cu_seqlens=s["cu"],
            chunk_states=kept, output_dinitial_state=True, **layer)
        return (out, final, dx, ddelta, dA, dB, dC, dD, dh0) + tuple(
            t for t in (dz, dbias) if t is not None)
    if op == "select":
        return gdn.beam_select(s["logits"], s["scores"], num_candidates=case["candidates"])
    return s["pool"], gdn.state_pool_reorder(s["pool"], s["idx"], s["parents"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op.startswith(("conv", "scan")):
        lens = _ints(case["lens"]) if "lens" in case else [1] * case["seqs"]
        n, tokens, c = len(lens), sum(lens), case["channels"]
        e, es, ss = tokens * c, SIZES[case["dtype"]], SIZES[case.get("state", "f32")]
    if op.startswith("conv"):
        w = case["width"]
        par = c * (w + (1 if case["bias"] else 0)) * SIZES[case["weight"]]
        rows = n * (w - 1) * c * ss
        if op != "conv training":
            return {"bytes": 2 * e * es + par + 2 * rows, "flops": 2 * w * e}
        # forward: x -> out; backward: x, dout -> dx; parameters and their gradients
        return {"bytes": 5 * e * es + 3 * par + 5 * rows, "flops": 8 * w * e}
    if op.startswith("scan"):
        ns = case["states"]
        rows, bc = n * c * ns * ss, 2 * tokens * case["groups"] * ns * es
        par, wide = 4 * c * (ns + 2), 4 if case["gated"] else 3
        if op != "scan training":
            # decay (product, exp), input, state, output of each state of a token
            return {"bytes": wide * e * es + bc + par + 2 * rows, "flops": 7 * e * ns}
        # backward: the inputs and dout again, a gradient of each input
        return {"bytes": (3 * wide - 1) * e * es + 3 * bc + 3 * par + 5 * rows,
                "flops": 28 * e * ns}
    if op == "select":
        rows, m = case["batch"] * case["beams"], case["candidates"]
        return {"bytes": rows * case["vocab"] * SIZES[case["dtype"]] + 12 * case["batch"] * m,
                "flops": 3 * rows * case["vocab"]}
    k = case["beams"]
    copies = case["batch"] * k * (1 - 1 / k) ** k  # beams without a child
    row = math.prod(_ints(case["row"])) * SIZES[case["to"]]
    return {"bytes": int(2 * copies * row) + 12 * case["batch"] * k, "flops": 0}


# --------------------------------------------------- the definitions, in fp64

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("conv"):
        return _exact_conv(s)
    if op.startswith("scan"):
        return _exact_scan(s)
    if op == "select":
        p = s["logits"].double()
        flat = (s["scores"].double()[:, :, None] + torch.log_softmax(p, -1)).reshape(p.shape[0], -1)
        return torch.sort(flat, dim=-1, descending=True).values[:, :case["candidates"]], None, None
    pool, parents = s["pool"].double(), s["parents"].tolist()
    before = pool.clone()
    for p, own_rows in zip(parents, s["idx"].reshape(len(parents), -1).tolist()):
        free = [r for i, r in enumerate(own_rows) if i not in p]
        for j, parent in enumerate(p):
            if parent in p[:j]:
                pool[free.pop(0)] = before[own_rows[parent]]
    return pool, None


def _exact_rows(s):
    return s["idx"].tolist() if "idx" in s else list(range(len(s["lens"])))


def _exact_conv(s):
    """Each sequence as a whole: its state and tokens, padded in front."""
    case, w = s["case"], s["w"].double()
    keep, training = case["width"] - 1, case["op"] == "conv training"
    out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    final = (s["final"] if "idx" in s else s["h0"]).double().clone()
    dx, dh0, t = torch.empty_like(out), torch.zeros_like(final), 0
    dw, db = torch.zeros_like(w), torch.zeros(case["channels"], dtype=torch.float64, device="cuda")
    bias = 0.0 if s["bias"] is None else s["bias"].double()
    for i, (r, n) in enumerate(zip(_exact_rows(s), s["lens"])):
        seen = torch.cat([s["h0"][r].double(), s["x"][t:t + n].double()])
        pre = bias + sum(seen[j:j + n] * w[:, j] for j in range(keep + 1))
        sig = 1 / (1 + torch.exp(-pre))
        out[t:t + n] = pre * sig if case["silu"] else pre
        final[r] = seen[n:]
        if training:
            d = s["dout"][t:t + n].double()
            if case["silu"]:
                d = d * (sig + pre * sig * (1 - sig))
            dseen = torch.zeros_like(seen)
            for j in range(keep + 1):
                dseen[j:j + n] += d * w[:, j]
                dw[:, j] += (d * seen[j:j + n]).sum(0)
            dseen[n:] += s["dfinal"][i].double()
            db += d.sum(0)
            dh0[i], dx[t:t + n] = dseen[:keep], dseen[keep:]
        t += n
    if not training:
        return out, final
    return (out, final, dx, dw, dh0) + (() if s["bias"] is None else (db,))


def _exact_scan(s):
    case = s["case"]
    training, c, g, ns = case["op"] == "scan training", case["channels"], case["groups"], case["states"]
    x, raw, A, D = s["x"].double(), s["delta"].double(), s["A"].double(), s["D"].double()
    tokens = x.shape[0]
    if training and tokens * c * ns > 2 ** 29:
        return None
    if s["dbias"] is not None:
        raw = raw + s["dbias"].double()
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())) if case["softplus"] else raw
    of = torch.arange(c, device="cuda") // (c // g)
    B, C = s["B"].double(), s["C"].double()
    y, final = torch.empty_like(x), (s["final"] if "idx" in s else s["h0"]).double().clone()
    hs = torch.empty((tokens, c, ns), dtype=torch.float64, device="cuda") if training else None
    t, begins = 0, []
    for r, n in zip(_exact_rows(s), s["lens"]):
        h = s["h0"][r].double()
        begins.append(t)
        for _ in range(n):
            h = torch.exp(dt[t, :, None] * A) * h + (dt[t] * x[t])[:, None] * B[t][of]
            y[t] = (h * C[t][of]).sum(-1)
            if training:
                hs[t] = h
            t += 1
        final[r] = h
    y += D * x
    z = s["z"].double() if case["gated"] else None
    sig = 1 / (1 + torch.exp(-z)) if case["gated"] else None
    out = y * z * sig if case["gated"] else y
    if not training:
        return out, final
    dout = s["dout"].double()
    dy = dout * z * sig if case["gated"] else dout
    dz = (dout * y * (sig + z * sig * (1 - sig)),) if case["gated"] else ()
    dx, ddt, dA = D * dy, torch.empty_like(x), torch.zeros_like(A)
    dB, dC, dh0 = torch.zeros_like(B), torch.zeros_like(C), torch.zeros_like(final)
    for i, (t0, n) in enumerate(zip(begins, s["lens"])):
        back = s["dfinal"][i].double()
        for t in range(t0 + n - 1, t0 - 1, -1):
            before = hs[t - 1] if t > t0 else s["h0"][i].double()
            dh = back + dy[t][:, None] * C[t][of]
            decay = torch.exp(dt[t, :, None] * A)
            dC[t].index_add_(0, of, dy[t][:, None] * hs[t])
            dB[t].index_add_(0, of, dh * (dt[t] * x[t])[:, None])
            du, da = (dh * B[t][of]).sum(-1), dh * before * decay
            dx[t] += du * dt[t]
            ddt[t] = du * x[t] + (da * A).sum(-1)
            dA += da * dt[t][:, None]
            back = decay * dh
        dh0[i] = back
    if case["softplus"]:
        ddt = ddt / (1 + torch.exp(-raw))
    grads = (dx, ddt, dA, dB, dC, (dy * x).sum(0), dh0) + dz
    return (out, final) + grads + (() if s["dbias"] is None else (ddt.sum(0),))
