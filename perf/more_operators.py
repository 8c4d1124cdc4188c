"""The cases by which the serving operators of a hybrid of gated-delta-rule and attention layers are measured: prompts
and single tokens of the gated delta rule, attention of a tree of drafted tokens over a paged cache, and the rows that
prompts and accepted drafts add to that cache."""
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
        # a chat turn appended to a cached state: latency counts
        {"name": "gdn_97_h32", "op": "gdn", "lens": "97", "H": 32, "G": 16, "dk": 128, "dv": 128, "dtype": "bf16",
         "init": True},
        # one ordinary prompt
        {"name": "gdn_2048_h32", "op": "gdn", "lens": "2048", "H": 32, "G": 16, "dk": 128, "dv": 128, "dtype": "bf16",
         "init": False},
        # a packed batch of unlike prompts, one of them a single token, resumed from cached states
        {"name": "gdn_ragged_h64", "op": "gdn", "lens": "2048,777,513,1", "H": 64, "G": 8, "dk": 128, "dv": 128,
         "dtype": "bf16", "init": True},
        # a long document
        {"name": "gdn_32768_h32", "op": "gdn", "lens": "32768", "H": 32, "G": 16, "dk": 128, "dv": 128, "dtype": "bf16",
         "init": False},
        # full precision, keys narrower than values, an empty sequence in the batch
        {"name": "gdn_f32_ragged", "op": "gdn", "lens": "300,0,1025", "H": 16, "G": 16, "dk": 64, "dv": 128,
         "dtype": "f32", "init": True},
        # one interactive user's next token
        {"name": "gdn_decode_1_h32", "op": "gdn_decode", "batch": 1, "H": 32, "G": 16, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # a full decode batch
        {"name": "gdn_decode_256_h64", "op": "gdn_decode", "batch": 256, "H": 64, "G": 8, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # one user's next token after a long document
        {"name": "attn_1x32768", "op": "attn", "lens": "32768", "T": 1, "H": 32, "KV": 8, "D": 128, "page": 64,
         "dtype": "bf16", "tree": False, "gaps": False},
        # a speculative step of a full batch: trees of 16 drafts
        {"name": "attn_64x4096_tree16", "op": "attn", "lens": ",".join(str(4096 - 29 * i) for i in range(64)), "T": 16,
         "H": 32, "KV": 8, "D": 128, "page": 64, "dtype": "bf16", "tree": True, "gaps": False},
        # full precision, small odd pages, a sequence without a past, places of the tree left empty
        {"name": "attn_f32_ragged_tree7", "op": "attn", "lens": "1000,0,77,513", "T": 7, "H": 12, "KV": 4, "D": 64,
         "page": 24, "dtype": "f32", "tree": True, "gaps": True},
        # the same packed prompts' keys and values into the pages
        {"name": "append_ragged", "op": "append", "lens": "2048,777,513,1", "past": 1000, "KV": 8, "D": 128, "page": 64,
         "dtype": "bf16"},
        # the accepted paths of a speculative step of a large batch
        {"name": "commit_256_t8", "op": "commit", "batch": 256, "T": 8, "past": 500, "KV": 8, "D": 128, "page": 64,
         "dtype": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def _draw_lens(rng, tokens, most):
    """Some lengths that add up to tokens, short, empty and long ones among them."""
    lens = []
    for _ in range(rng.randint(0, most)):
        lens.append(min(tokens // 2, rng.choice([0, 1, _log_uniform(rng, 1, 2048)])))
        tokens -= lens[-1]
    lens.append(tokens)
    rng.shuffle(lens)
    return ",".join(str(n) for n in lens)


def draw(rng):
    op = rng.choice(["gdn", "gdn", "gdn", "gdn_decode", "attn", "attn", "attn", "append", "commit"])
    if op in ("gdn", "gdn_decode"):
        G = rng.choice([1, 2, 4, 8, 16])
        case = {"op": op, "H": G * rng.choice([1, 2, 4]), "G": G, "dk": rng.choice([64, 128, 128]),
                "dv": rng.choice([64, 128, 128]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "gdn_decode":
            return {**case, "batch": _log_uniform(rng, 1, 256)}
        tokens = _log_uniform(rng, 1, min(32768, 32768 * 32 // case["H"]) if case["dtype"] == "bf16" else 4096)
        return {**case, "lens": _draw_lens(rng, tokens, 5), "init": rng.random() < 0.5}
    kv = {"KV": rng.choice([1, 2, 4, 8]), "D": rng.choice([64, 128, 128]), "page": rng.choice([1, 16, 24, 64, 64, 128, 500]),
          "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "append":
        return {"op": op, "lens": _draw_lens(rng, _log_uniform(rng, 1, 8192), 5), "past": rng.randint(0, 1000), **kv}
    if op == "commit":
        return {"op": op, "batch": _log_uniform(rng, 1, 256), "T": rng.choice([1, 2, 4, 8, 16, 61]),
                "past": rng.randint(0, 1000), **kv}
    T, H = rng.choice([1, 1, 2, 4, 7, 16, 33, 64]), kv["KV"] * rng.choice([1, 2, 4, 5, 8])
    bf16 = kv["dtype"] == "bf16"
    tokens = _log_uniform(rng, 16, min(131072 if bf16 else 32768, (1 << (27 if bf16 else 24)) // (H * T)))
    lens = [min(tokens // 2, rng.choice([0, 1, _log_uniform(rng, 1, 4096)])) for _ in range(_log_uniform(rng, 1, 32) - 1)]
    lens.append(max(0, min(32768, tokens - sum(lens))))
    rng.shuffle(lens)
    return {"op": op, "lens": ",".join(str(n) for n in lens), "T": T, "H": H, **kv, "tree": rng.random() < 0.6,
            "gaps": rng.random() < 0.3}


# ---- inputs --------------------------------------------------------------------------------------
def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _gdn_tokens(gen, tokens, case):
    """Queries and keys of unit norm; gates exp(-a softplus(x)) and write strengths sigmoid(x) as such layers have
    them after initialisation, a in [1, 16] and softplus(x) around 0.001 to 0.1."""
    dt, d, H = _DTYPES[case["dtype"]], {"device": "cuda", "generator": gen}, case["H"]
    q, k = (torch.randn(tokens, case["G"], case["dk"], **d) for _ in range(2))
    q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
    v = torch.randn(tokens, H, case["dv"], **d)
    a = 1 + 15 * torch.rand(H, **d)
    bias = torch.log(torch.expm1(torch.exp(torch.rand(H, **d) * math.log(100.0) + math.log(1e-3))))
    x = torch.randn(tokens, H, **d) + bias
    g = -a * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
    beta = 1 / (1 + torch.exp(-torch.randn(tokens, H, **d)))
    return {"q": q.to(dt), "k": k.to(dt), "v": v.to(dt), "g": g, "beta": beta}


def _pool(gen, lens, case):
    """Pages of a cache in the midst of serving: every slot's pages scattered over the pool, one page to spare."""
    page, dt = case["page"], _DTYPES[case["dtype"]]
    per = max(1, -(-max(lens) // page))
    npages = len(lens) * per + 1
    shape = (npages, page, case["KV"], case["D"])
    k, v = (torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32).to(dt) for _ in range(2))
    order = torch.randperm(npages, device="cuda", generator=gen)[: len(lens) * per]
    return {"k_pages": k, "v_pages": v, "table": order.to(torch.int32).view(len(lens), per).contiguous()}


def _tree(gen, S, T, tree, gaps):
    """The parent of each draft: -1 follows the last token of the past, -2 is an empty place."""
    own_place = torch.arange(T, device="cuda").expand(S, T)
    parent = own_place - 1
    if tree:   # one of the drafts before, rather a late one
        near = torch.rand(S, T, device="cuda", generator=gen).square()
        parent = torch.floor((own_place + 1) * (1 - near)).long().clamp(max=T) - 1
        parent = torch.minimum(parent, own_place - 1)
    if gaps:   # empty places at the end, and one row of nothing else
        count = (torch.rand(S, device="cuda", generator=gen) * (T + 1)).long()
        parent = torch.where(own_place < count[:, None], parent, -2)
    return parent.to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"op": op}
    if op == "gdn":
        lens = _lens(case)
        state.update(_gdn_tokens(gen, sum(lens), case), max_len=max(lens), scale=case["dk"] ** -0.5, init=None)
        state["cu"] = _ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        if case["init"]:
            state["init"] = torch.randn(len(lens), case["H"], case["dv"], case["dk"], device="cuda", generator=gen) * 0.3
        return state
    if op == "gdn_decode":
        B, npages = case["batch"], case["batch"] + 3
        state.update(_gdn_tokens(gen, B, case), scale=case["dk"] ** -0.5)
        pool = torch.randn(npages, case["H"], case["dv"], case["dk"], device="cuda", generator=gen) * 0.3
        page = torch.randperm(npages, device="cuda", generator=gen)[:B].to(torch.int32)
        state.update(pool=pool, page=page)
        if own:  # the cache that a serving program keeps
            cache = _ers().LinAttnCache(B, case["H"], case["G"], case["dk"], case["dv"], npages=npages,
                                        io_dtype=_DTYPES[case["dtype"]], state=pool)
            cache.pages.table.copy_(page.view(B, 1))
            state["cache"] = cache
        return state
    dt, KV, D = _DTYPES[case["dtype"]], case["KV"], case["D"]
    new = {"device": "cuda", "generator": gen}
    if op == "attn":
        lens, T = _lens(case), case["T"]
        S = len(lens)
        state.update(_pool(gen, lens, case), pos=_ints(lens), scale=D ** -0.5, max_len=max(lens))
        state["q"] = (torch.randn(S, T, case["H"], D, **new) * 2).to(dt)
        state["k"], state["v"] = (torch.randn(S, T, KV, D, **new).to(dt) for _ in range(2))
        state["parent"] = _tree(gen, S, T, case["tree"], case["gaps"]) if case["tree"] or case["gaps"] else None
        # what a page holds behind its sequence's last token is left over from other sequences
        past = torch.arange(state["table"].shape[1] * case["page"], device="cuda")
        behind = (past >= state["pos"][:, None]).view(S, -1, case["page"])
        for name in ("k_pages", "v_pages"):
            pages = state[name]
            rows = pages[state["table"].long()]
            pages[state["table"].long()] = rows.masked_fill_(behind[..., None, None], math.nan)
    else:
        lens = _lens(case) if op == "append" else [case["T"]] * case["batch"]
        S = len(lens)
        start = torch.randint(0, case["past"] + 1, (S,), **new).to(torch.int32)
        state.update(_pool(gen, [case["past"] + n for n in lens], case), start=start, pos=start.clone())
        shape = (sum(lens), KV, D) if op == "append" else (S, case["T"], KV, D)
        state["k"], state["v"] = (torch.randn(shape, **new).to(dt) for _ in range(2))
        if op == "append":
            state["cu"] = _ints([sum(lens[:i]) for i in range(S + 1)])
        else:      # the accepted drafts of each sequence, in the order of their path through the tree
            state["accepted"] = _ints([_accepted(case, i) for i in range(S)])
            path = torch.rand(S, case["T"], **new).argsort(1)
            live = torch.arange(case["T"], device="cuda") < state["accepted"][:, None]
            state["path"] = torch.where(live, path, case["T"]).sort(1).values.to(torch.int32)
    if own:  # the cache that a serving program keeps
        table = state["table"]
        cache = _ers().AttnCache(table.shape[0], KV, D, page_tokens=case["page"], slot_pages=table.shape[1],
                                 npages=state["k_pages"].shape[0], io_dtype=dt, k=state["k_pages"], v=state["v_pages"])
        cache.pages.table.copy_(table)
        cache.pages.refs[table.flatten().long()] = 1
        cache.pos.copy_(state["pos"])
        state["cache"] = cache
    return state


def _accepted(case, i):
    return (5 * i + 3) % (case["T"] + 1)


# ---- plain forms ---------------------------------------------------------------------------------
def _plain_gdn(s):
    """Chunks of 64 tokens over sequences padded to whole chunks.  Inside a chunk the residuals solve a unit lower
    triangular system, whose inverse is a product of powers; from chunk to chunk the state is multiplied by a matrix
    and gains another, and these pairs are joined by doubling."""
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"].long()
    T, G, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    S, C = cu.numel() - 1, 64
    n = max(1, -(-s["max_len"] // C))
    pos = torch.arange(n * C, device=q.device)
    length = cu[1:] - cu[:-1]
    live = pos < length[:, None]
    index = torch.where(live, cu[:-1, None] + pos, 0)

    def spread(x):
        y = x[index] if T else x.new_zeros(S, n * C, *x.shape[1:])
        y = torch.where(live[..., None, None], y.float(), 0.0).movedim(2, 1)
        return y.repeat_interleave(H // x.shape[1], 1).view(S, H, n, C, -1)

    qf, kf, vf, beta = spread(q), spread(k), spread(v), spread(s["beta"][..., None])
    gate = spread(s["g"][..., None])[..., 0].double().cumsum(-1)          # from the chunk's start
    i = torch.arange(C, device=q.device)
    gap = gate[..., :, None] - gate[..., None, :]
    decay = torch.where(i[:, None] >= i, torch.exp(gap.clamp(max=0)).float(), 0.0)
    since, left = torch.exp(gate).float()[..., None], torch.exp(gate[..., -1:] - gate).float()[..., None]
    one = torch.eye(C, device=q.device)
    x1 = torch.where(i[:, None] > i, -beta * decay * (kf @ kf.transpose(-1, -2)), 0.0)
    x2 = x1 @ x1
    x4 = x2 @ x2
    x8 = x4 @ x4
    x16 = x8 @ x8
    inverse = (one + x1) @ (one + x2) @ (one + x4) @ (one + x8) @ (one + x16) @ (one + x16 @ x16)
    w, u0 = inverse @ (beta * since * kf), inverse @ (beta * vf)
    turn = since[..., -1:, :] * torch.eye(dk, device=q.device) - w.transpose(-1, -2) @ (left * kf)
    gain = u0.transpose(-1, -2) @ (left * kf)
    step = 1
    while step < n:  # turn and gain of the chunks up to each one
        gain = torch.cat([gain[:, :, :step], gain[:, :, :-step] @ turn[:, :, step:] + gain[:, :, step:]], 2)
        turn = torch.cat([turn[:, :, :step], turn[:, :, :-step] @ turn[:, :, step:]], 2)
        step *= 2
    init = s["init"] if s["init"] is not None else torch.zeros(S, H, dv, dk, device=q.device)
    after = init[:, :, None] @ turn + gain
    before = torch.cat([init[:, :, None], after[:, :, :-1]], 2)
    u = u0 - w @ before.transpose(-1, -2)
    o = since * (qf @ before.transpose(-1, -2)) + (decay * (qf @ kf.transpose(-1, -2))) @ u
    o = (o * s["scale"]).view(S, H, n * C, dv).movedim(1, 2)
    seq = torch.bucketize(torch.arange(T, device=q.device), cu[1:], right=True)
    o = o[seq, torch.arange(T, device=q.device) - cu[seq]]
    return {"o": o.to(v.dtype), "state": after[:, :, -1]}


def _plain_gdn_decode(s):
    q, k, v, page = s["q"], s["k"], s["v"], s["page"].long()
    H, G = v.shape[1], q.shape[1]
    qf, kf = (x.float().repeat_interleave(H // G, 1)[:, :, None] for x in (q, k))
    state = s["pool"][page] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (v.float() - (state * kf).sum(-1))
    state = state + u[..., None] * kf
    s["pool"][page] = state
    return {"o": ((state * qf).sum(-1) * s["scale"]).to(v.dtype), "pool": s["pool"]}


def _plain_attn(s):
    q, pos = s["q"], s["pos"].long()
    S, T, H, D = q.shape
    page, KV = s["k_pages"].shape[1:3]
    L = s["max_len"]
    at = torch.arange(L, device=q.device)
    live = at < pos[:, None]
    rows = s["table"].long()[:, at // page] * page + at % page if L else at.expand(S, L)

    def all_of(pages, drafts):
        past = torch.where(live[..., None, None], pages.view(-1, KV, D)[rows].float(), 0.0)
        return torch.cat([past, drafts.float()], 1).movedim(2, 1)          # [S, KV, L + T, D]

    place = torch.arange(T, device=q.device)
    parent = s["parent"].long() if s["parent"] is not None else (place - 1).expand(S, T)
    there = parent > -2
    seen = ((parent[..., None] == place) | (place[:, None] == place)).float()
    seen = seen @ seen      # the draft, its parent and the one before, then four, eight, ... of the path
    seen = seen @ seen
    seen = seen.clamp(max=1) @ seen.clamp(max=1)
    seen = seen.clamp(max=1) @ seen.clamp(max=1)
    seen = seen.clamp(max=1) @ seen.clamp(max=1)
    seen = (seen.clamp(max=1) @ seen.clamp(max=1) > 0) & there[:, None]
    seen = torch.cat([live[:, None].expand(S, T, L), seen], 2) & there[..., None]
    qf = q.float().view(S, T, KV, H // KV, D).permute(0, 2, 1, 3, 4).reshape(S, KV, T * (H // KV), D)
    x = (qf @ all_of(s["k_pages"], s["k"]).transpose(-1, -2)).view(S, KV, T, H // KV, L + T) * s["scale"]
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    top = x.max(-1, keepdim=True).values
    e = torch.exp(x - torch.where(top == -math.inf, 0.0, top)).view(S, KV, -1, L + T)
    total = e.sum(-1, keepdim=True)
    o = (e @ all_of(s["v_pages"], s["v"])) / torch.where(total > 0, total, 1.0)
    return o.view(S, KV, T, H // KV, D).permute(0, 2, 1, 3, 4).reshape(S, T, H, D).to(q.dtype)


def _plain_rows(s, seq, position, source):
    """Row `source` of the new keys and values goes to its sequence's `position`."""
    page, KV, D = s["k_pages"].shape[1:]
    to = s["table"].long()[seq, position // page] * page + position % page
    s["k_pages"].view(-1, KV, D)[to] = s["k"].view(-1, KV, D)[source]
    s["v_pages"].view(-1, KV, D)[to] = s["v"].view(-1, KV, D)[source]


def _plain_append(s):
    cu, pos = s["cu"].long(), s["pos"].long()
    row = torch.arange(s["k"].shape[0], device=cu.device)
    seq = torch.bucketize(row, cu[1:], right=True)
    _plain_rows(s, seq, pos[seq] + row - cu[seq], row)
    s["pos"] += (cu[1:] - cu[:-1]).to(torch.int32)


def _plain_commit(s):
    pos, path = s["pos"].long(), s["path"].long()
    S, T = path.shape
    seq, n = torch.nonzero(torch.arange(T, device=path.device) < s["accepted"][:, None], as_tuple=True)
    _plain_rows(s, seq, pos[seq] + n, seq * T + path[seq, n])
    s["pos"] += s["accepted"]


def run(s):
    op = s["op"]
    if not own:
        if op == "gdn":
            return _plain_gdn(s)
        if op == "gdn_decode":
            return _plain_gdn_decode(s)
        if op == "attn":
            return _plain_attn(s)
        s["pos"].copy_(s["start"])      # every pass adds the same rows
        if op == "append":
            _plain_append(s)
        else:
            _plain_commit(s)
        return {"k": s["k_pages"], "v": s["v_pages"], "pos": s["pos"]}
    ers = _ers()
    if op == "gdn":
        o, state = ers.gdn_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"], init_state=s["init"],
                               scale=s["scale"], max_seqlen=s["max_len"], check=False)
        return {"o": o, "state": state}
    cache = s["cache"]
    if op == "gdn_decode":
        o = ers.gdn_decode(cache, s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], check=False)
        return {"o": o, "pool": cache.state}
    if op == "attn":
        return ers.attn_verify(cache, s["q"], s["k"], s["v"], parent=s["parent"], scale=s["scale"],
                               max_len=s["max_len"], check=False)
    cache.pos.copy_(s["start"])
    if op == "append":
        ers.attn_append(cache, s["k"], s["v"], cu_seqlens=s["cu"], check=False)
    else:
        ers.attn_commit(cache, s["k"], s["v"], s["accepted"], path=s["path"], check=False)
    return {"k": cache.k, "v": cache.v, "pos": cache.pos}


# ---- the work that no implementation can leave out -----------------------------------------------
def work(case):
    op, b = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("gdn", "gdn_decode"):
        lens = _lens(case) if op == "gdn" else [1] * case["batch"]
        state = case["H"] * case["dk"] * case["dv"]
        reads = 1 if op == "gdn_decode" or case["init"] else 0
        tokens = sum(lens)
        return {"bytes": tokens * (2 * (case["G"] * case["dk"] + case["H"] * case["dv"]) * b + 8 * case["H"])
                + (1 + reads) * len(lens) * state * 4,
                "flops": 6 * state * tokens}
    row = case["KV"] * case["D"] * b
    if op == "attn":
        lens, T = _lens(case), case["T"]
        q = case["H"] * case["D"]
        return {"bytes": 2 * (sum(lens) + len(lens) * T) * row + 2 * len(lens) * T * q * b,
                "flops": 4 * q * T * sum(lens) + 2 * q * T * (T + 1) * len(lens)}
    rows = sum(_lens(case)) if op == "append" else sum(_accepted(case, i) for i in range(case["batch"]))
    return {"bytes": 4 * rows * row + 8, "flops": 0}


# ---- the definitions, in 64 bits -----------------------------------------------------------------
def _delta_rule(q, k, v, g, beta, state, scale):
    """One token: S <- e^g S, S <- S + beta (v - S k) k^T, o = scale S q, for [..., dv, dk] states."""
    state = state * torch.exp(g)[..., None, None]
    u = beta[..., None] * (v - (state @ k[..., None])[..., 0])
    state = state + u[..., :, None] * k[..., None, :]
    return state, (state @ q[..., None])[..., 0] * scale


def exact(case, seed):
    op = case["op"]
    if op in ("append", "commit"):  # rows are copied, not computed
        return None
    s = prepare(case, seed)
    if op == "attn":
        S, T, H, D = s["q"].shape
        KV, out = case["KV"], torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        parents = s["parent"].tolist() if s["parent"] is not None else [list(range(-1, T - 1))] * S
        for i, n in enumerate(_lens(case)):
            pages = s["table"][i, : -(-n // case["page"])].long()
            past = [s[x][pages].double().reshape(-1, KV, D)[:n] for x in ("k_pages", "v_pages")]
            k, v = (torch.cat([a, s[x][i].double()]) for a, x in zip(past, ("k", "v")))
            seen = torch.zeros(T, n + T, dtype=torch.bool)
            for t, p in enumerate(parents[i]):
                if p == -2:
                    continue
                seen[t, :n] = True
                if p >= 0:
                    seen[t] |= seen[p]
                seen[t, n + t] = True
            seen = seen.cuda()
            for h in range(H):
                x = s["q"][i, :, h].double() @ k[:, h // (H // KV)].T * s["scale"]
                x = x.masked_fill(~seen, -math.inf)
                p = torch.where(seen.any(1, keepdim=True), torch.softmax(x, -1), torch.zeros_like(x))
                out[i, :, h] = p @ v[:, h // (H // KV)]
        return out
    H = case["H"]
    group = torch.arange(H, device="cuda") // (H // case["G"])
    if op == "gdn_decode":
        pool = s["pool"].double()
        at = s["page"].long()
        state, o = _delta_rule(s["q"].double()[:, group], s["k"].double()[:, group], s["v"].double(), s["g"].double(),
                               s["beta"].double(), pool[at], s["scale"])
        pool[at] = state
        return {"o": o, "pool": pool}
    lens = _lens(case)
    o = torch.zeros(sum(lens), H, case["dv"], dtype=torch.float64, device="cuda")
    finals, at = [], 0
    for i, n in enumerate(lens):
        state = torch.zeros(H, case["dv"], case["dk"], dtype=torch.float64, device="cuda")
        if s["init"] is not None:
            state = s["init"][i].double()
        for t in range(at, at + n):
            state, o[t] = _delta_rule(s["q"][t, group].double(), s["k"][t, group].double(), s["v"][t].double(),
                                      s["g"][t].double(), s["beta"][t].double(), state, s["scale"])
        finals.append(state)
        at += n
    return {"o": o, "state": torch.stack(finals)}
