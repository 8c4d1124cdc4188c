"""The cases by which the serving operators around a linear-attention layer are measured: prompts and
single tokens of linear attention with a decay per head, the pages of its state cache, and the log
probabilities by which its branches are scored."""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ers():
    import exact_replay_decode_gb300 as ers
    return ers


# ---- the cases -----------------------------------------------------------------------------------
def listed():
    return [
        # the shortest useful prompt (a chat turn appended to a cached state): latency counts
        {"name": "prefill_97_h32", "op": "prefill", "lens": "97", "H": 32, "G": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "init": True},
        # one ordinary prompt
        {"name": "prefill_2048_h32", "op": "prefill", "lens": "2048", "H": 32, "G": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "init": False},
        # a packed batch of unlike prompts, one of them a single token, resumed from cached states
        {"name": "prefill_ragged_h64", "op": "prefill", "lens": "2048,777,513,1", "H": 64, "G": 8, "dk": 128,
         "dv": 128, "dtype": "bf16", "init": True},
        # a long document
        {"name": "prefill_32768_h32", "op": "prefill", "lens": "32768", "H": 32, "G": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "init": False},
        # full precision, keys narrower than values, an empty sequence in the batch
        {"name": "prefill_f32_ragged", "op": "prefill", "lens": "300,0,1025", "H": 16, "G": 16, "dk": 64, "dv": 128,
         "dtype": "f32", "init": True},
        # one interactive user's next token
        {"name": "decode_1_h32", "op": "decode", "batch": 1, "H": 32, "G": 16, "dk": 128, "dv": 128, "dtype": "bf16"},
        # a full decode batch
        {"name": "decode_256_h64", "op": "decode", "batch": 256, "H": 64, "G": 8, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # one prompt branched into eight samples, each given a state of its own
        {"name": "pages_fork_1x8", "op": "fork", "parents": 1, "children": 8, "slot_pages": 1, "spare": 7,
         "page": 524288, "side": 0},
        # a serving cache after an eighth of its sequences ended, and then another eighth: compacted both times
        {"name": "pages_compact_256", "op": "compact", "slots": 256, "freed": 32, "slot_pages": 1, "spare": 17,
         "page": 524288, "side": 0},
        # scoring one sampled token over an odd vocabulary
        {"name": "logprobs_1x50001", "op": "logprobs", "rows": 1, "vocab": 50001, "pad": 0, "k": 8, "dtype": "bf16",
         "masked": 0.0, "scale": 1.0},
        # scoring the drafts of a speculative step: 512 sequences x 4 drafts
        {"name": "logprobs_2048x131072", "op": "logprobs", "rows": 2048, "vocab": 131072, "pad": 0, "k": 20,
         "dtype": "bf16", "masked": 0.0, "scale": 1.0},
        # full precision under a grammar's mask that leaves some rows nothing, rows padded, tempered
        {"name": "logprobs_515x32000_masked", "op": "logprobs", "rows": 515, "vocab": 32000, "pad": 64, "k": 5,
         "dtype": "f32", "masked": 0.9, "scale": 1.25},
    ]


def _log_uniform(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    return n - 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "fork", "compact", "logprobs", "logprobs"])
    if op in ("prefill", "decode"):
        G = rng.choice([1, 2, 4, 8, 16])
        case = {"op": op, "H": G * rng.choice([1, 2, 4]), "G": G, "dk": rng.choice([64, 128, 128]),
                "dv": rng.choice([64, 128, 128]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "decode":
            return {**case, "batch": _log_uniform(rng, 1, 256)}
        tokens = _log_uniform(rng, 1, min(32768, 32768 * 32 // case["H"]) if case["dtype"] == "bf16" else 4096)
        lens = []
        for _ in range(rng.randint(0, 5)):
            lens.append(min(tokens // 2, rng.choice([0, 1, _log_uniform(rng, 1, 2048)])))
            tokens -= lens[-1]
        lens.append(tokens)
        rng.shuffle(lens)
        return {**case, "lens": ",".join(str(n - (n == 3072)) for n in lens), "init": rng.random() < 0.5}
    if op == "fork":
        return {"op": op, "parents": _log_uniform(rng, 1, 12), "children": rng.randint(1, 8),
                "slot_pages": rng.choice([1, 1, 2, 4]), "spare": rng.randint(1, 30),
                "page": 4 * _log_uniform(rng, 64, 131072), "side": rng.choice([0, 0, 24, 1001])}
    if op == "compact":
        slots = _log_uniform(rng, 4, 256)
        return {"op": op, "slots": slots, "freed": rng.randint(1, slots // 2), "slot_pages": rng.choice([1, 1, 2]),
                "spare": rng.randint(1, 30), "page": 4 * _log_uniform(rng, 64, 65536), "side": rng.choice([0, 0, 24, 1001])}
    vocab = _log_uniform(rng, 1000, 131072)
    return {"op": op, "rows": _log_uniform(rng, 1, min(2048, 134217728 // vocab)), "vocab": vocab,
            "pad": rng.choice([0, 0, 1, 64]), "k": rng.choice([0, 1, 5, 20, 32]),
            "dtype": rng.choice(["bf16", "bf16", "f32"]), "masked": rng.choice([0.0, 0.0, 0.5, 0.99]),
            "scale": rng.choice([1.0, 1.0, 0.7, 1.4])}


# ---- inputs --------------------------------------------------------------------------------------
def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _log_decay(H):
    """Per-head slopes from 0.84 down to 1/256, as layers with a fixed decay per head spread them."""
    return -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32, device="cuda") / H)


def _qkv(gen, tokens, case):
    """Activations with unit-norm-sized queries and keys."""
    dt, d = _DTYPES[case["dtype"]], {"device": "cuda", "generator": gen}
    q = (torch.randn(tokens, case["G"], case["dk"], **d) * case["dk"] ** -0.5).to(dt)
    k = (torch.randn(tokens, case["G"], case["dk"], **d) * case["dk"] ** -0.5).to(dt)
    v = torch.randn(tokens, case["H"], case["dv"], **d).to(dt)
    return q, k, v


def _pages_state(case, gen, nslots):
    """A pool in the midst of serving: every slot owns its pages, scattered over the pool."""
    per = case["slot_pages"]
    npages = nslots * per + case["spare"]
    arrays = [torch.randn(npages, case["page"], device="cuda", generator=gen)]
    if case["side"]:
        arrays.append(torch.randn(npages, case["side"], device="cuda", generator=gen).to(torch.bfloat16))
    order = torch.randperm(npages, device="cuda", generator=gen)[: nslots * per]
    table = order.to(torch.int32).view(nslots, per).contiguous()
    refs = torch.zeros(npages, dtype=torch.int32, device="cuda")
    refs[order] = 1
    return {"arrays": arrays, "table": table, "refs": refs}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"op": op}
    if op == "prefill":
        lens = _lens(case)
        q, k, v = _qkv(gen, sum(lens), case)
        cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        init = None
        if case["init"]:
            init = torch.randn(len(lens), case["H"], case["dv"], case["dk"], device="cuda", generator=gen) * 0.3
        state.update(q=q, k=k, v=v, log_decay=_log_decay(case["H"]), cu=cu, max_len=max(lens), init=init,
                     scale=1.0)
    elif op == "decode":
        B = case["batch"]
        q, k, v = _qkv(gen, B, case)
        npages = B + 3
        pool = torch.randn(npages, case["H"], case["dv"], case["dk"], device="cuda", generator=gen) * 0.3
        page = torch.randperm(npages, device="cuda", generator=gen)[:B].to(torch.int32)
        state.update(q=q, k=k, v=v, log_decay=_log_decay(case["H"]), pool=pool, page=page, scale=1.0)
        if own:  # the cache that a serving program keeps
            cache = _ers().LinAttnCache(B, case["H"], case["G"], case["dk"], case["dv"], npages=npages,
                                        io_dtype=_DTYPES[case["dtype"]], state=pool)
            cache.pages.table.copy_(page.view(B, 1))
            state["cache"] = cache
    elif op == "fork":
        P, C = case["parents"], case["children"]
        state.update(_pages_state(case, gen, P * (1 + C)))
        state["child"] = torch.arange(P, P * (1 + C), dtype=torch.int32, device="cuda")
        state["parent"] = torch.arange(P, dtype=torch.int32, device="cuda").repeat_interleave(C)
    elif op == "compact":
        n, f = case["slots"], case["freed"]
        state.update(_pages_state(case, gen, n))
        slots = torch.randperm(n, device="cuda", generator=gen).to(torch.int32)
        state.update(first=slots[:f].clone(), second=slots[f:2 * f].clone())
    else:
        R, V, pad = case["rows"], case["vocab"], case["pad"]
        full = torch.randn(R, V + pad, device="cuda", generator=gen) * 3.0
        full[:, ::7] += 1.5
        if case["masked"]:
            full.masked_fill_(torch.rand(R, V + pad, device="cuda", generator=gen) < case["masked"], -math.inf)
            full[::37] = -math.inf
            full[5::41, : V // 2] = torch.finfo(_DTYPES[case["dtype"]]).min
        full = full.to(_DTYPES[case["dtype"]])
        target = torch.randint(0, V, (R,), device="cuda", generator=gen).to(torch.int32)
        target[7::11] = -1
        state.update(logits=full[:, :V], target=target, k=case["k"], scale=case["scale"])
    if own and op in ("fork", "compact"):  # the pool that a serving program keeps
        state["pool"] = _ers().PagePool(state["arrays"], state["table"], state["refs"])
    return state


# ---- plain forms ---------------------------------------------------------------------------------
def _plain_prefill(s):
    """Chunks of 128 tokens over sequences padded to whole chunks: masked products inside a chunk, the
    states before each chunk as one product with the matrix of decays between chunks."""
    q, k, v, a, cu = s["q"], s["k"], s["v"], s["log_decay"], s["cu"].long()
    T, G, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    S, C = cu.numel() - 1, 128
    n = max(1, -(-s["max_len"] // C))
    pos = torch.arange(n * C, device=q.device)
    length = cu[1:] - cu[:-1]
    live = pos < length[:, None]
    index = torch.where(live, cu[:-1, None] + pos, 0)

    def spread(x):
        y = x[index] if T else x.new_zeros(S, n * C, *x.shape[1:])
        y = torch.where(live[..., None, None], y.float(), 0.0).movedim(2, 1)
        return y.repeat_interleave(H // x.shape[1], 1).view(S, H, n, C, -1)

    qf, kf, vf = spread(q), spread(k), spread(v)
    init = s["init"] if s["init"] is not None else torch.zeros(S, H, dv, dk, device=q.device)
    i = torch.arange(C, device=q.device)
    gap = i[:, None] - i
    inside = torch.where(gap >= 0, torch.exp(a[:, None, None] * gap.clamp(min=0)), 0.0)
    o = (qf @ kf.transpose(-1, -2) * inside[:, None]) @ vf
    ends = torch.exp(a[:, None] * (C - 1 - i))
    local = (vf * ends[:, None, :, None]).transpose(-1, -2) @ kf
    c = torch.arange(n, device=q.device)
    apart = c[:, None] - 1 - c
    between = torch.where(apart >= 0, torch.exp(a[:, None, None] * C * apart.clamp(min=0)), 0.0)
    before = (between @ local.view(S, H, n, dv * dk)).view(S, H, n, dv, dk)
    before = before + torch.exp(a[:, None] * C * c)[:, :, None, None] * init[:, :, None]
    o = o + (qf @ before.transpose(-1, -2)) * torch.exp(a[:, None] * (i + 1))[:, None, :, None]
    o = (o * s["scale"]).view(S, H, n * C, dv).movedim(1, 2)
    seq = torch.bucketize(torch.arange(T, device=q.device), cu[1:], right=True)
    o = o[seq, torch.arange(T, device=q.device) - cu[seq]]
    left = (length[:, None] - 1 - pos).clamp(min=0)
    weight = torch.where(live[:, None], torch.exp(a[:, None] * left[:, None]), 0.0)
    final = (vf.view(S, H, n * C, dv) * weight[..., None]).transpose(-1, -2) @ kf.view(S, H, n * C, dk)
    final = final + torch.exp(a * length[:, None])[..., None, None] * init
    return {"o": o.to(v.dtype), "state": final}


def _plain_decode(s):
    q, k, v, page = s["q"], s["k"], s["v"], s["page"].long()
    H, G = v.shape[1], q.shape[1]
    qf, kf = (x.float().repeat_interleave(H // G, 1) for x in (q, k))
    state = s["pool"][page] * torch.exp(s["log_decay"])[:, None, None] + v.float()[..., None] * kf[:, :, None]
    s["pool"][page] = state
    o = (state * qf[:, :, None]).sum(-1) * s["scale"]
    return {"o": o.to(v.dtype), "pool": s["pool"]}


def _plain_free(s, slots):
    table, refs, at = s["table"], s["refs"], slots.long()
    old = table[at].flatten()
    refs.index_add_(0, old.clamp(min=0).long(), -(old >= 0).to(torch.int32))
    table[at] = -1


def _plain_fork(s, src, dst):
    table, refs = s["table"], s["refs"]
    rows = table[src.long()]
    table[dst.long()] = rows
    rows = rows.flatten()
    refs.index_add_(0, rows.clamp(min=0).long(), (rows >= 0).to(torch.int32))


def _plain_own(s, slots, copy):
    """Every page of the slots that is shared or missing becomes a page of their own, lowest free page first."""
    table, refs, at = s["table"], s["refs"], slots.long()
    old = table[at].flatten()
    held = old.clamp(min=0).long()
    need = (old < 0) | (refs[held] > 1)
    free = torch.sort((refs > 0).to(torch.int32), stable=True).indices
    new = torch.where(need, free[(need.cumsum(0) - 1).clamp(min=0)], held)
    refs.index_add_(0, held, -(need & (old >= 0)).to(torch.int32))
    refs.index_add_(0, new, need.to(torch.int32))
    table[at] = new.to(torch.int32).view(at.numel(), -1)
    if copy:
        for x in s["arrays"]:
            x[new] = torch.where((old < 0)[:, None], torch.zeros_like(x[:1]), x[held])
    return old.view(at.numel(), -1)


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    ids = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    count = live.sum()
    mover, hole = live & (ids >= count), ~live & (ids < count)
    holes = torch.sort((~hole).to(torch.int32), stable=True).indices
    to = torch.where(mover, holes[(mover.cumsum(0) - 1).clamp(min=0)], ids)
    source = torch.cat([ids, ids[:1]]).scatter_(0, torch.where(mover, to, refs.numel()), ids)[:-1]
    for x in s["arrays"]:
        x.copy_(x[source])
    remap = torch.where(live, to, -1).to(torch.int32)
    refs.copy_(torch.where(ids < count, refs[source], 0))
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], -1))
    return remap, count.to(torch.int32).view(1)


def _plain_logprobs(s):
    logits, target, k = s["logits"], s["target"].long(), s["k"]
    R, V = logits.shape
    x = logits.float()
    top = x.max(1).values
    empty = top == -math.inf
    d = (x - torch.where(empty, 0.0, top)[:, None]) * s["scale"]
    e = torch.exp(d)
    total = torch.where(empty, 1.0, e.sum(1))
    log_total = torch.log(total)
    entropy = log_total - (e * torch.where(e > 0, d, 0.0)).sum(1) / total
    picked = d.gather(1, target.clamp(min=0)[:, None])[:, 0] - log_total
    logprob = torch.where(target < 0, 0.0, torch.where(empty, -math.inf, picked))
    entropy = torch.where(empty, 0.0, entropy)
    # the order of (value, then lowest index) as one whole number
    bits = (logits.float() + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 32) + (V - 1 - torch.arange(V, device=x.device))
    best = key.topk(k, dim=1).indices
    best_d = d.gather(1, best)
    gone = x.gather(1, best) == -math.inf
    return {"logprob": logprob, "entropy": entropy, "top_id": torch.where(gone, -1, best).to(torch.int32),
            "top_logprob": torch.where(gone, -math.inf, best_d - log_total[:, None])}


def _pool_of(s):
    return {"table": s["table"], "refs": s["refs"], "arrays": s["arrays"]}


def run(s):
    op = s["op"]
    if not own:
        if op == "prefill":
            return _plain_prefill(s)
        if op == "decode":
            return _plain_decode(s)
        if op == "fork":
            _plain_free(s, s["child"])
            _plain_fork(s, s["parent"], s["child"])
            return {"read": _plain_own(s, s["child"], True), **_pool_of(s)}
        if op == "compact":
            _plain_free(s, s["first"])
            one = _plain_compact(s)
            _plain_own(s, s["first"], False)
            _plain_free(s, s["second"])
            two = _plain_compact(s)
            _plain_own(s, s["second"], False)
            return {"remap": [one[0], two[0]], "live": [one[1], two[1]], **_pool_of(s)}
        return _plain_logprobs(s)
    ers = _ers()
    if op == "prefill":
        o, state = ers.linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], cu_seqlens=s["cu"], init_state=s["init"],
                                   scale=s["scale"], max_seqlen=s["max_len"], check=False)
        return {"o": o, "state": state}
    if op == "decode":
        o = ers.linattn_decode(s["cache"], s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], check=False)
        return {"o": o, "pool": s["cache"].state}
    if op == "fork":
        ers.pages_free(s["pool"], s["child"], check=False)
        ers.pages_fork(s["pool"], s["parent"], s["child"], check=False)
        return {"read": ers.pages_own(s["pool"], s["child"], copy=True, check=False), **_pool_of(s)}
    if op == "compact":
        ers.pages_free(s["pool"], s["first"], check=False)
        one = ers.pages_compact(s["pool"], check=False)
        ers.pages_own(s["pool"], s["first"], copy=False, check=False)
        ers.pages_free(s["pool"], s["second"], check=False)
        two = ers.pages_compact(s["pool"], check=False)
        ers.pages_own(s["pool"], s["second"], copy=False, check=False)
        return {"remap": [one[0], two[0]], "live": [one[1], two[1]], **_pool_of(s)}
    logprob, entropy, top_id, top_logprob = ers.token_logprobs(s["logits"], s["target"], top_k=s["k"],
                                                               scale=s["scale"], check=False)
    return {"logprob": logprob, "entropy": entropy, "top_id": top_id, "top_logprob": top_logprob}


# ---- the work that no implementation can leave out -----------------------------------------------
def work(case):
    op = case["op"]
    if op in ("prefill", "decode"):
        b = 2 if case["dtype"] == "bf16" else 4
        lens = _lens(case) if op == "prefill" else [1] * case["batch"]
        state = case["H"] * case["dk"] * case["dv"]
        reads = 1 if op == "decode" or case["init"] else 0
        tokens = sum(lens)
        return {"bytes": tokens * 2 * (case["G"] * case["dk"] + case["H"] * case["dv"]) * b
                + (1 + reads) * len(lens) * state * 4 + 4 * case["H"],
                "flops": 4 * state * tokens}
    if op in ("fork", "compact"):
        page = case["page"] * 4 + case["side"] * 2
        per = case["slot_pages"]
        if op == "fork":  # each parent's pages read once, each child's written
            slots, moved = case["parents"] * (1 + case["children"]), per * case["parents"] * (1 + case["children"])
        else:             # in the steady state, one page read and one written for each freed page, twice
            slots, moved = case["slots"], 4 * per * case["freed"]
        return {"bytes": moved * page + 8 * (2 * slots * per + case["spare"]), "flops": 0}
    b = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["rows"] * (case["vocab"] * b + 12 + 8 * case["k"]), "flops": 5 * case["rows"] * case["vocab"]}


# ---- the definitions, in 64 bits -----------------------------------------------------------------
def _recurrence(q, k, v, a, state, scale):
    """One token: S <- e^a S + v k^T, o = scale S q, for [..., H, dv, dk] states."""
    state = state * torch.exp(a)[:, None, None] + v[..., :, None] * k[..., None, :]
    return state, (state @ q[..., None])[..., 0] * scale


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):  # pages are copied, not computed
        return None
    s = prepare(case, seed)
    if op == "logprobs":
        logps, entropies, tops = [], [], []
        for i in range(0, case["rows"], 64):
            x = s["logits"][i:i + 64].double()
            x = (x - x.max(1, keepdim=True).values) * s["scale"]  # a row of lowest values is an even one
            t = s["target"][i:i + 64].long()
            lp = x - torch.logsumexp(x, 1, keepdim=True)
            # rows that the mask leaves nothing, and what 32 bits do not reach
            lp = torch.where(torch.isnan(lp) | (lp < -torch.finfo(torch.float32).max), torch.full_like(lp, -math.inf), lp)
            logps.append(torch.where(t < 0, torch.zeros_like(x[:, 0]), lp.gather(1, t.clamp(min=0)[:, None])[:, 0]))
            entropies.append(-torch.where(lp == -math.inf, torch.zeros_like(lp), lp.exp() * lp).sum(1))
            tops.append(lp.topk(case["k"], dim=1).values)
        return {"logprob": torch.cat(logps), "entropy": torch.cat(entropies), "top_id": None,
                "top_logprob": torch.cat(tops)}
    H, G = case["H"], case["G"]
    a = s["log_decay"].double()
    group = torch.arange(H, device="cuda") // (H // G)
    if op == "decode":
        pool = s["pool"].double()
        state, o = _recurrence(s["q"].double()[:, group], s["k"].double()[:, group], s["v"].double(), a,
                               pool[s["page"].long()], s["scale"])
        pool[s["page"].long()] = state
        return {"o": o, "pool": pool}
    lens = _lens(case)
    o = torch.zeros(sum(lens), H, case["dv"], dtype=torch.float64, device="cuda")
    finals, at = [], 0
    for i, n in enumerate(lens):
        state = torch.zeros(H, case["dv"], case["dk"], dtype=torch.float64, device="cuda")
        if s["init"] is not None:
            state = s["init"][i].double()
        for t in range(at, at + n):
            state, o[t] = _recurrence(s["q"][t, group].double(), s["k"][t, group].double(), s["v"][t].double(), a,
                                      state, s["scale"])
        finals.append(state)
        at += n
    return {"o": o, "state": torch.stack(finals)}
