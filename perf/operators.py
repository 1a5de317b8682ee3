"""Cases and plain forms of the operators of a continuous-batching step: request tables, packed convolution, headed scan.

Five operators, of a server (or a packed trainer's forward) that runs requests of different lengths without padding:

  tables      block table and slot map from request lengths
  conv        short causal convolution over packed prompts, with a cache of windows by slot
  conv_step   the same for one token per request
  scan        selective scan with one decay per head over packed prompts, with a cache of states by slot
  scan_step   the same for one token per request
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def listed():
    return [
        # a decode batch with two prompts that have just come in
        {"name": "tables_decode", "op": "tables", "requests": 66, "tokens": 1100, "block": 256, "skew": "decode"},
        # a large prefill batch: many requests, long and short
        {"name": "tables_prefill", "op": "tables", "requests": 1000, "tokens": 200000, "block": 512, "skew": "ragged"},
        # eight prompts of 2048 in front of a 24-head layer: x, B and C pass the convolution together
        {"name": "conv_prompt", "op": "conv", "requests": 8, "tokens": 16384, "dim": 1792, "width": 4, "dtype": "bf16", "skew": "even", "pad": 0},
        # odd sizes in fp32: rows that no vector load fits, a batch padded at its end
        {"name": "conv_odd_fp32", "op": "conv", "requests": 37, "tokens": 2999, "dim": 1023, "width": 3, "dtype": "fp32", "skew": "ragged", "pad": 57},
        # four users at once: latency
        {"name": "conv_step_few", "op": "conv_step", "requests": 4, "dim": 1792, "width": 4, "dtype": "bf16"},
        # a full decode batch of a wide layer
        {"name": "conv_step_many", "op": "conv_step", "requests": 512, "dim": 5376, "width": 4, "dtype": "bf16"},
        # eight prompts of 2048 through a 24-head layer with the gate
        {"name": "scan_prompt", "op": "scan", "requests": 8, "tokens": 16384, "heads": 24, "groups": 1, "headdim": 64, "dstate": 128, "dtype": "bf16", "z": True, "skew": "even", "pad": 0},
        # one long document: the sequence is all there is to split
        {"name": "scan_long", "op": "scan", "requests": 1, "tokens": 65536, "heads": 32, "groups": 1, "headdim": 64, "dstate": 128, "dtype": "bf16", "z": False, "skew": "even", "pad": 0},
        # prompts of 1 to some hundred tokens, two groups, half precision, a padded batch
        {"name": "scan_ragged_fp16", "op": "scan", "requests": 40, "tokens": 6001, "heads": 16, "groups": 2, "headdim": 64, "dstate": 64, "dtype": "fp16", "z": True, "skew": "ragged", "pad": 23},
        # odd head sizes in fp32
        {"name": "scan_odd_fp32", "op": "scan", "requests": 5, "tokens": 777, "heads": 6, "groups": 3, "headdim": 40, "dstate": 24, "dtype": "fp32", "z": False, "skew": "ragged", "pad": 0},
        # one user's next token
        {"name": "scan_step_one", "op": "scan_step", "requests": 1, "heads": 24, "groups": 1, "headdim": 64, "dstate": 128, "dtype": "bf16", "z": True},
        # a full decode batch of an 80-head layer
        {"name": "scan_step_many", "op": "scan_step", "requests": 256, "heads": 80, "groups": 8, "headdim": 64, "dstate": 128, "dtype": "bf16", "z": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["tables", "conv", "conv_step", "scan", "scan", "scan", "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp32"])
    skew = rng.choice(["even", "ragged", "ragged", "decode"])
    if op == "tables":
        r = _log(rng, 1, 2048)
        return {"op": op, "requests": r, "tokens": _log(rng, r, 200000), "block": 128 * rng.randint(1, 16), "skew": skew}
    if op == "conv":
        r = _log(rng, 1, 64)
        return {"op": op, "requests": r, "tokens": _log(rng, r, 16384), "dim": _log(rng, 8, 1800), "width": rng.randint(2, 4), "dtype": dtype, "skew": skew, "pad": rng.choice([0, 0, 31])}
    if op == "conv_step":
        return {"op": op, "requests": _log(rng, 1, 512), "dim": _log(rng, 8, 5376), "width": rng.randint(2, 4), "dtype": dtype}
    groups = rng.choice([1, 1, 2, 3])
    heads = groups * rng.randint(1, 24 // groups)
    headdim, dstate = rng.choice([64, 64, 64, 128, 32, 40, 80, 17]), rng.choice([128, 128, 64, 16, 72, 96, 33])
    shape = {"heads": heads, "groups": groups, "headdim": headdim, "dstate": dstate, "dtype": dtype, "z": rng.random() < 0.5}
    if op == "scan":
        r = _log(rng, 1, 64)
        return {"op": op, "requests": r, "tokens": _log(rng, r, 4096 if dtype == "fp32" else 16384), **shape, "skew": skew, "pad": rng.choice([0, 0, 31])}
    return {"op": op, "requests": _log(rng, 1, 256), **shape}


def _lengths(case, rng):
    """Request lengths that sum to the case's tokens; a ragged batch of more than four holds one empty request."""
    r, t = case["requests"], case["tokens"]
    if case["skew"] == "even":
        n = np.full(r, t // r)
        n[: t % r] += 1
    elif case["skew"] == "decode":  # one token each, and the rest in one or two prompts
        n = np.minimum(np.ones(r, np.int64), t)
        rest = t - int(n.sum())
        n[int(rng.integers(r))] += rest - rest // 3
        n[int(rng.integers(r))] += rest // 3
    else:
        cut = np.sort(rng.integers(0, t + 1, r - 1))
        n = np.diff(np.concatenate([[0], cut, [t]]))
        if r > 4:
            k = int(rng.integers(r - 1))
            n[k + 1] += n[k]
            n[k] = 0
    return n.astype(np.int32)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000 + seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _head_inputs(case, g, rows):
    t = _TYPES[case["dtype"]]
    h, p, n, k = case["heads"], case["headdim"], case["dstate"], case["groups"]
    # what the projection and the convolution leave: x, B and C side by side in one row, dt and z beside them
    xbc = _normal(g, (rows, h * p + 2 * k * n), t)
    s = {"x": xbc[:, : h * p].view(rows, h, p), "B": xbc[:, h * p : h * p + k * n].view(rows, k, n), "C": xbc[:, h * p + k * n :].view(rows, k, n)}
    s["dt"] = _normal(g, (rows, h), t)
    s["z"] = _normal(g, (rows, h, p), t) if case["z"] else None
    s["A"] = -(1 + 15 * torch.rand(h, generator=g, device="cuda"))
    s["D"] = 1 + 0.1 * torch.randn(h, generator=g, device="cuda")
    first = 0.001 + 0.099 * torch.rand(h, generator=g, device="cuda")
    s["dt_bias"] = torch.log(torch.expm1(first))
    return s


def _slots(rng, requests, spare):
    """Slots of the requests in a cache with some spare ones, in no order."""
    return torch.from_numpy(rng.permutation(requests + spare)[:requests].astype(np.int32)).cuda()


def prepare(case, seed):
    rng, g, op, r = np.random.default_rng(seed), _gen(seed), case["op"], case["requests"]
    s = {"case": case}
    if op in ("tables", "conv", "scan"):
        n = _lengths(case, rng)
        s["tokens"] = case["tokens"] + case.get("pad", 0)
        s["lengths"] = torch.from_numpy(n).cuda()
        # half of the requests go on from an earlier chunk
        s["context"] = torch.from_numpy((rng.integers(0, 2, r) * rng.integers(1, 5000, r)).astype(np.int32)).cuda()
    if op == "tables":
        s["slots"] = torch.where(s["context"] > 0, _slots(rng, r, 8), -1).to(torch.int32)
        s["free"] = torch.from_numpy((r + 8 + rng.permutation(r)).astype(np.int32)).cuda()
        return s
    s["slots"] = _slots(rng, r, 3)
    if op in ("conv", "conv_step"):
        t, d, w = _TYPES[case["dtype"]], case["dim"], case["width"]
        s["x"] = _normal(g, (s["tokens"] if op == "conv" else r, d), t)
        s["weight"] = _normal(g, (d, w), torch.float32, 0.5)
        s["bias"] = _normal(g, (d,), torch.float32, 0.1)
        s["state"] = _normal(g, (r + 3, d, w - 1), t)
    else:
        s |= _head_inputs(case, g, s["tokens"] if op == "scan" else r)
        s["state"] = _normal(g, (r + 3, case["heads"], case["headdim"], case["dstate"]), torch.float32, 0.5)
    if own and op in ("conv", "scan"):
        from state_space_model_03_gb300 import head_scan_block, request_tables

        block = head_scan_block(s["tokens"], r, case["heads"], case["headdim"], dtype=s["x"].dtype) if op == "scan" else 512
        s["tables"] = request_tables(s["lengths"], s["tokens"], context=s["context"], slots=s["slots"], block=block)
    return s


# ---- plain forms -----------------------------------------------------------------------------------------------------


def _owner(starts, n):
    """For 0..n-1, the last row whose start is not past it (starts ascend; empty rows share a start)."""
    marks = torch.zeros(n + 1, dtype=torch.int64, device=starts.device)
    marks.index_add_(0, starts.long().clamp(max=n), torch.ones_like(starts, dtype=torch.int64))
    return torch.cumsum(marks[:n], 0) - 1


def _offsets(lengths):
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=lengths.device), torch.cumsum(lengths, 0)])


def _block_table(lengths, tokens, block):
    """Rows (request, first token, tokens, index in the request), (-1, 0, 0, 0) past the last; and how many there are."""
    r = lengths.numel()
    most = tokens // block + min(r, tokens)
    off = _offsets(lengths)
    per = _offsets((lengths + block - 1) // block)
    i = torch.arange(most, device=lengths.device)
    req = _owner(per[:-1], most)
    k = i - per[req]
    row = torch.stack([req, off[req] + k * block, torch.clamp(lengths[req] - k * block, max=block), k], 1)
    blank = torch.tensor([-1, 0, 0, 0], device=lengths.device)
    return torch.where((i < per[-1])[:, None], row, blank), per[-1]


def _plain_tables(s):
    n, tokens = s["lengths"], s["tokens"]
    off = _offsets(n)
    i = torch.arange(tokens, device=n.device)
    req = _owner(off[:-1], tokens)
    live = i < off[-1]
    new = s["slots"] < 0
    rank = torch.cumsum(new, 0) - 1
    table, blocks = _block_table(n, tokens, s["case"]["block"])
    out = {
        "offsets": off,
        "token_request": torch.where(live, req, -1),
        "token_position": torch.where(live, s["context"][req] + i - off[req], 0),
        "blocks": table,
        "slots": torch.where(new, s["free"][rank.clamp(min=0)], s["slots"]),
        "counts": torch.stack([off[-1], blocks, new.sum(), torch.zeros_like(blocks)]),
    }
    return {k: v.to(torch.int32) for k, v in out.items()}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_conv(s):
    x, w, st = s["x"].float(), s["weight"], s["state"]
    t, h = x.shape[0], w.shape[1] - 1
    off = _offsets(s["lengths"])
    i = torch.arange(t, device=x.device)
    req = _owner(off[:-1], t)
    pos = i - off[req]
    # the windows that the requests start from, oldest first: (requests, width - 1, dim)
    start = torch.where((s["context"] > 0)[:, None, None], st[s["slots"].long()].float(), 0.0).transpose(1, 2)
    # rows of [all windows, all tokens]; tap k of token t is the token k-h places before it, or a row of its window
    rows = torch.cat([start.reshape(-1, x.shape[1]), x])
    k = torch.arange(h + 1, device=x.device) - h
    at = torch.where(pos[:, None] + k >= 0, start.shape[0] * h + i[:, None] + k, req[:, None] * h + pos[:, None] + k + h)
    acc = (rows[at] * w.t()).sum(1) + s["bias"]
    out = torch.where((i < off[-1])[:, None], _silu(acc), 0.0).to(s["x"].dtype)
    n = s["lengths"][:, None].long()
    last = torch.arange(h, device=x.device) - h
    r = torch.arange(n.shape[0], device=x.device)[:, None]
    at = torch.where(n + last >= 0, start.shape[0] * h + off[:-1, None] + n + last, r * h + n + last + h)
    new = rows[at].transpose(1, 2).to(st.dtype)
    keep = (n > 0)[:, :, None]
    st[s["slots"].long()] = torch.where(keep, new, st[s["slots"].long()])
    return {"out": out, "state": st}


def _plain_conv_step(s):
    st, at = s["state"], s["slots"].long()
    win = torch.cat([st[at], s["x"][:, :, None]], 2)
    out = _silu((win.float() * s["weight"]).sum(2) + s["bias"]).to(s["x"].dtype)
    st[at] = win[:, :, 1:]
    return {"out": out, "state": st}


def _sums_between(v):
    """sums[..., i, j] = v[..., j+1] + ... + v[..., i] for j <= i, else -inf."""
    n = v.shape[-1]
    low = torch.tril(torch.ones(n, n, dtype=torch.bool, device=v.device), -1)
    part = torch.cumsum(torch.where(low, v[..., :, None], 0.0), -2)
    return torch.where(torch.tril(torch.ones_like(low)), part, -math.inf)


def _plain_scan(s, chunk=64):
    """Products inside chunks of 64 tokens, and one product over the chunks of each request for the states between them."""
    x, b, c, st = s["x"].float(), s["B"].float(), s["C"].float(), s["state"]
    t, h, p = x.shape
    rep = h // b.shape[1]
    table, _ = _block_table(s["lengths"], t, chunk)
    req, first, size, index = table.unbind(1)
    j = torch.arange(chunk, device=x.device)
    live = j < size[:, None]
    at = torch.where(live, first[:, None] + j, 0)
    dt = torch.where(live[:, :, None], _softplus(s["dt"][at].float() + s["dt_bias"]), 0.0)
    xs = torch.where(live[:, :, None, None], x[at], 0.0) * dt[..., None]
    bs, cs = (torch.where(live[:, :, None, None], v[at], 0.0) for v in (b, c))
    a = (dt * s["A"]).transpose(1, 2)  # (chunks, heads, tokens)
    inside = torch.exp(_sums_between(a))
    score = torch.einsum("kign,kjgn->kgij", cs, bs).repeat_interleave(rep, 1) * inside
    y = torch.einsum("khij,kjhp->kihp", score, xs)
    gained = torch.einsum("khj,kjhp,kjhn->khpn", inside[:, :, -1], xs, bs.repeat_interleave(rep, 2))
    # the state before each chunk: the request's start, and what its earlier chunks gained, each with the decay since
    total = torch.where((req >= 0)[:, None], a.sum(-1), 0.0)
    past = _sums_between(total.t())  # (heads, i, j): decays of chunks j+1 .. i
    same = req[:, None] == req[None, :]
    fade = torch.where(same, torch.exp(past), 0.0)
    after = torch.einsum("hij,jhpn->ihpn", fade, gained)
    slots = s["slots"].long()
    start = torch.where((s["context"] > 0)[:, None, None, None], st[slots], 0.0)
    own_first = torch.arange(table.shape[0], device=x.device) - index
    whole = torch.exp(past[:, torch.arange(table.shape[0], device=x.device), own_first].t() + total[own_first])
    after = after + whole[..., None, None] * start[req.clamp(min=0)]
    before = torch.where((index > 0)[:, None, None, None], after.roll(1, 0), start[req.clamp(min=0)])
    since = torch.exp(torch.cumsum(a, -1)).transpose(1, 2)
    y = y + torch.einsum("kihn,khpn->kihp", cs.repeat_interleave(rep, 2), before) * since[..., None]
    y = y + s["D"][:, None] * torch.where(live[:, :, None, None], x[at], 0.0)
    if s["z"] is not None:
        y = y * _silu(s["z"][at].float())
    out = torch.zeros((t + 1, h, p), device=x.device)
    out[torch.where(live, first[:, None] + j, t)] = y
    n = s["lengths"]
    end = torch.cumsum((n + chunk - 1) // chunk, 0) - 1
    st[slots] = torch.where((n > 0)[:, None, None, None], after[end.clamp(min=0)], st[slots])
    return {"out": out[:t].to(s["x"].dtype), "state": st}


def _plain_scan_step(s):
    x, st, at = s["x"].float(), s["state"], s["slots"].long()
    rep = x.shape[1] // s["B"].shape[1]
    b, c = (v.float().repeat_interleave(rep, 1) for v in (s["B"], s["C"]))
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    new = torch.exp(dt * s["A"])[..., None, None] * st[at] + (dt[..., None] * x)[..., None] * b[:, :, None, :]
    y = (new * c[:, :, None, :]).sum(-1) + s["D"][:, None] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    st[at] = new
    return {"out": y.to(s["x"].dtype), "state": st}


_PLAIN = {"tables": _plain_tables, "conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_step": _plain_scan_step}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    import state_space_model_03_gb300 as ssm

    if op == "tables":
        t = ssm.request_tables(s["lengths"], s["tokens"], context=s["context"], slots=s["slots"], free_slots=s["free"], block=s["case"]["block"])
        return {"offsets": t.offsets, "token_request": t.token_request, "token_position": t.token_position, "blocks": t.blocks, "slots": t.slots, "counts": t.counts}
    if op == "conv":
        out = ssm.packed_conv1d_fn(s["x"], s["weight"], s["tables"], bias=s["bias"], conv_state=s["state"], activation="silu")
    elif op == "conv_step":
        out = ssm.packed_conv1d_update(s["x"], s["state"], s["weight"], bias=s["bias"], slots=s["slots"], activation="silu")
    elif op == "scan":
        out = ssm.head_scan_fn(s["x"], s["dt"], s["A"], s["B"], s["C"], s["tables"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, state=s["state"])
    else:
        out = ssm.head_state_update(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, slots=s["slots"])
    return {"out": out, "state": s["state"]}


# ---- work ------------------------------------------------------------------------------------------------------------


def work(case):
    op, r = case["op"], case["requests"]
    t = case["tokens"] + case.get("pad", 0) if "tokens" in case else r
    if op == "tables":
        rows = t // case["block"] + min(r, t)
        return {"bytes": 4 * (3 * r + r // 2) + 4 * (2 * t + 2 * r + 1 + 4 * rows + 4), "flops": 2 * t}
    e = _SIZE[case["dtype"]]
    if op in ("conv", "conv_step"):
        d, w = case["dim"], case["width"]
        kept = (1.5 if op == "conv" else 2) * r * d * (w - 1) * e
        return {"bytes": int(2 * t * d * e + kept + 4 * d * (w + 1)), "flops": 2 * t * d * (w + 2)}
    h, p, n, g = case["heads"], case["headdim"], case["dstate"], case["groups"]
    rows = t * e * ((3 if case["z"] else 2) * h * p + h + 2 * g * n)
    states = (1.5 if op == "scan" else 2) * 4 * r * h * p * n
    # the recurrence itself: one product-sum into each state and one out of it
    return {"bytes": int(rows + states + 12 * h), "flops": t * h * (4 * p * n + 6 * p)}


# ---- in 64 bits, from the definitions --------------------------------------------------------------------------------


def _exact_tables(s):
    lens, ctx, slots, free = (s[k].cpu().numpy().astype(np.int64) for k in ("lengths", "context", "slots", "free"))
    t, block = s["tokens"], s["case"]["block"]
    off, owner, place, rows, got, taken = [0], np.full(t, -1), np.zeros(t, np.int64), [], [], 0
    for r, n in enumerate(lens):
        o = off[-1]
        owner[o : o + n] = r
        place[o : o + n] = ctx[r] + np.arange(n)
        rows += [(r, o + k, min(block, n - k), k // block) for k in range(0, n, block)]
        off.append(o + n)
        got.append(slots[r] if slots[r] >= 0 else free[taken])
        taken += slots[r] < 0
    most = t // block + min(len(lens), t)
    table = np.array(rows + [(-1, 0, 0, 0)] * (most - len(rows))).reshape(most, 4)
    found = {"offsets": off, "token_request": owner, "token_position": place, "blocks": table, "slots": got, "counts": [off[-1], len(rows), taken, 0]}
    return {k: torch.from_numpy(np.asarray(v).astype(np.int32)) for k, v in found.items()}


def _exact_conv(s, single):
    x, w, bias, st = (s[k].double() for k in ("x", "weight", "bias", "state"))
    h = w.shape[1] - 1
    lens = [1] * x.shape[0] if single else s["lengths"].tolist()
    goes_on = [True] * x.shape[0] if single else (s["context"] > 0).tolist()
    out, at = torch.zeros_like(x), 0
    for n, slot, on in zip(lens, s["slots"].tolist(), goes_on):
        if n == 0:
            continue
        old = st[slot] if on else torch.zeros_like(st[slot])
        line = torch.cat([old, x[at : at + n].t()], 1)  # (dim, width - 1 + n)
        v = bias[:, None] + sum(w[:, k : k + 1] * line[:, k : k + n] for k in range(h + 1))
        out[at : at + n] = (v * torch.sigmoid(v)).t()
        st[slot] = line[:, n:]
        at += n
    return {"out": out, "state": st}


def _exact_scan(s, single):
    """Token by token, all requests side by side."""
    x, dt, a, d, bias, st = (s[k].double() for k in ("x", "dt", "A", "D", "dt_bias", "state"))
    rep = x.shape[1] // s["B"].shape[1]
    dt = torch.nn.functional.softplus(dt + bias, threshold=700.0)
    rows = x.shape[0]
    lens = [1] * rows if single else s["lengths"].tolist()
    firsts = torch.tensor(np.concatenate([[0], np.cumsum(lens)[:-1]]), device=x.device)
    # longest first, so that the requests that still have tokens are the first rows
    order = sorted(range(len(lens)), key=lambda r: -lens[r])
    at, slots = firsts[order], s["slots"].long()[order]
    goes_on = torch.ones(len(lens), dtype=torch.bool, device=x.device) if single else (s["context"] > 0)
    cur = st[slots] * goes_on[order][:, None, None, None]
    y = torch.zeros_like(x)
    keep = torch.exp(dt * a)
    live = len(lens)
    for i in range(lens[order[0]]):
        while lens[order[live - 1]] <= i:
            live -= 1
        k = at[:live] + i
        b, c = (s[n][k].double().repeat_interleave(rep, 1) for n in ("B", "C"))
        v = cur[:live]
        v.mul_(keep[k][:, :, None, None]).add_((dt[k][:, :, None] * x[k])[..., None] * b[:, :, None, :])
        y[k] = torch.matmul(v, c[..., None])[..., 0]
    used = sum(n > 0 for n in lens)
    st[slots[:used]] = cur[:used]
    y = y + d[:, None] * x
    y[sum(lens) :] = 0
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z * torch.sigmoid(z)
    return {"out": y, "state": st}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "tables":
        return _exact_tables(s)
    return (_exact_conv if op.startswith("conv") else _exact_scan)(s, op.endswith("step"))
