"""What is measured of attention with modified scores and of drafted trees over the cache.

With the scaled product x = q_i . k_j / sqrt(D) of a row at position i and a key at
position j, the score is

    s = cap tanh(x / cap) - slope_h |i - j|

(either part may be absent).  Key j is visible to row i from i - window on and up
to i (causal) or to the end, or, with a prefix, wherever j < prefix of its sample.
Cases: the forward on whole sequences, fixed length or packed; a training step
(forward, then the gradients); new tokens over a paged cache; a tree of drafted
tokens over the cache, where a bit per pair says which drafted tokens a row sees
(the window is for the tokens before them);
and the move of an accepted path's rows to the slots behind the context.

``run`` computes a case in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where ``own`` is true, through the library's entry
points.  ``exact`` gives the same outputs from the definitions in 64 bits.

Layouts: [B, H, S, D] with K and V of H_kv heads, or packed [T, H, D] with offsets;
the cache is [pages, page_size, H_kv, D] for K and for V, a block table of page
numbers per sequence, and a length per sequence that counts the new tokens.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- cases
# cap: 0 = none; bias: slopes 2^(-8 (h + 1) / H); window: -1 = unlimited, else keys before the row;
# gain: standard deviation of the scaled products; spread: how much shorter the shortest sequence may be.
def listed():
    return [
        # A prompt of a model with capped scores, 8 query heads to a K/V head of 128.
        {"name": "prompt_cap_gqa_d128", "op": "forward", "packed": False, "dtype": "bf16", "batch": 2, "len": 4096,
         "spread": 0, "H": 32, "H_kv": 4, "D": 128, "causal": True, "window": -1, "cap": 50.0, "bias": False,
         "prefix": 0, "gain": 4.0},
        # The library's benchmark shape with a bias that grows with distance in place of rotated positions.
        {"name": "prompt_bias_d64", "op": "forward", "packed": False, "dtype": "fp16", "batch": 4, "len": 4096,
         "spread": 0, "H": 16, "H_kv": 16, "D": 64, "causal": True, "window": -1, "cap": 0.0, "bias": True,
         "prefix": 0, "gain": 1.0},
        # Documents of mixed lengths, the first part of each seen by all of it; scores well into the cap.
        {"name": "prefix_packed_d64", "op": "forward", "packed": True, "dtype": "bf16", "batch": 7, "len": 2500,
         "spread": 2400, "H": 16, "H_kv": 2, "D": 64, "causal": True, "window": -1, "cap": 30.0, "bias": False,
         "prefix": 700, "gain": 8.0},
        # The smallest: a short odd batch with a local window, cap and bias together.
        {"name": "short_window_d32", "op": "forward", "packed": False, "dtype": "fp16", "batch": 3, "len": 257,
         "spread": 0, "H": 9, "H_kv": 3, "D": 32, "causal": True, "window": 100, "cap": 20.0, "bias": True,
         "prefix": 0, "gain": 3.0},
        # A training step with capped scores.
        {"name": "train_cap_gqa_d128", "op": "train", "packed": False, "dtype": "bf16", "batch": 1, "len": 4096,
         "spread": 0, "H": 32, "H_kv": 4, "D": 128, "causal": True, "window": -1, "cap": 50.0, "bias": False,
         "prefix": 0, "gain": 4.0},
        # A training step of an encoder on documents of mixed lengths, distance to both sides.
        {"name": "train_bias_packed_d64", "op": "train", "packed": True, "dtype": "fp16", "batch": 9, "len": 2047,
         "spread": 1700, "H": 16, "H_kv": 16, "D": 64, "causal": False, "window": -1, "cap": 0.0, "bias": True,
         "prefix": 0, "gain": 1.0},
        # A decoding step with capped scores: 32 sequences of mixed lengths.
        {"name": "decode_cap_b32", "op": "paged", "dtype": "bf16", "batch": 32, "q_len": 1, "q_spread": 0, "ctx": 8192,
         "spread": 7000, "H": 32, "H_kv": 4, "D": 128, "page": 64, "window": -1, "cap": 50.0, "bias": False,
         "gain": 4.0},
        # Chunks of prompts beside single tokens, with a local window, cap and bias.
        {"name": "chunk_window_d64", "op": "paged", "dtype": "fp16", "batch": 5, "q_len": 1500, "q_spread": 1499,
         "ctx": 8192, "spread": 3001, "H": 16, "H_kv": 4, "D": 64, "page": 16, "window": 4095, "cap": 30.0,
         "bias": True, "gain": 3.0},
        # Trees of up to 64 drafted tokens for 16 sequences.
        {"name": "tree_b16_d128", "op": "tree", "dtype": "bf16", "batch": 16, "q_len": 64, "q_spread": 40, "ctx": 8192,
         "spread": 6001, "H": 32, "H_kv": 4, "D": 128, "page": 64, "window": -1, "cap": 0.0, "bias": False,
         "gain": 1.0, "width": 3},
        # A small tree of one sequence; scores capped and biased.
        {"name": "tree_b1_d64", "op": "tree", "dtype": "fp16", "batch": 1, "q_len": 13, "q_spread": 0, "ctx": 2051,
         "spread": 0, "H": 16, "H_kv": 2, "D": 64, "page": 16, "window": -1, "cap": 30.0, "bias": True, "gain": 3.0,
         "width": 2},
        # Accepted paths of 48 sequences' trees, up to 9 tokens each.
        {"name": "keep_b48", "op": "keep", "dtype": "bf16", "batch": 48, "q_len": 64, "q_spread": 30, "ctx": 1024,
         "spread": 900, "H_kv": 8, "D": 128, "page": 16, "accept": 9},
        # An accepted path of one sequence.
        {"name": "keep_b1", "op": "keep", "dtype": "fp16", "batch": 1, "q_len": 13, "q_spread": 0, "ctx": 777,
         "spread": 0, "H_kv": 2, "D": 64, "page": 32, "accept": 4},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "train", "train", "paged", "paged", "tree", "tree", "keep"])
    D = rng.choice([16, 32, 64, 64, 128, 128])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    H = H_kv * rng.choice([1, 2, 3, 4, 5, 8] if H_kv <= 4 else [1, 2, 4])
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"])}
    if op == "keep":
        case["batch"] = _log_int(rng, 1, 64)
        case["q_len"] = _log_int(rng, 2, 120)
        case["q_spread"] = rng.randint(0, case["q_len"] - 1)
        case["ctx"] = case["q_len"] + _log_int(rng, 1, 40000 // case["batch"])
        case["spread"] = rng.randint(0, case["ctx"] - case["q_len"])
        case.update(H_kv=H_kv, D=D, page=rng.choice([16, 32, 64, 128]), accept=rng.randint(1, min(12, case["q_len"])))
        return case
    case.update(H=H, H_kv=H_kv, D=D, gain=rng.choice([1.0, 3.0, 8.0]))
    case["cap"] = rng.choice([0.0, 15.0, 30.0, 50.0])
    case["bias"] = rng.random() < 0.5 if case["cap"] or op == "tree" else True
    if op in ("forward", "train"):
        case["packed"] = rng.random() < 0.5
        case["batch"] = _log_int(rng, 1, 8)
        most = math.sqrt((2.0e11 if op == "forward" else 6.0e10) / (4.0 * D * H * case["batch"]))
        case["len"] = _log_int(rng, 1, min(8192, int(most)))
        case["spread"] = rng.randint(0, case["len"] - 1) if case["packed"] else 0
        case["causal"] = rng.random() < 0.7
        case["window"] = rng.choice([-1, -1, _log_int(rng, 1, case["len"])])
        case["prefix"] = rng.choice([0, rng.randint(1, case["len"])]) if case["causal"] else 0
        return case
    case["page"] = rng.choice([16, 32, 64, 128, 256])
    case["window"] = rng.choice([-1, -1, 0])
    if op == "tree":
        case["batch"] = _log_int(rng, 1, 32)
        case["q_len"] = _log_int(rng, 1, 100)
        case["width"] = rng.randint(1, 5)
        case["ctx"] = case["q_len"] + _log_int(rng, 1, min(32768, int(5.0e7 / (case["batch"] * H_kv * D))))
    elif rng.random() < 0.5:  # single tokens
        case["batch"] = _log_int(rng, 1, 64)
        case["q_len"] = 1 if rng.random() < 0.6 else rng.randint(2, 8)
        case["ctx"] = case["q_len"] + _log_int(rng, 1, min(131072, int(1.4e8 / (case["batch"] * H_kv * D))))
    else:                     # chunks
        case["batch"] = _log_int(rng, 1, 8)
        case["q_len"] = _log_int(rng, 9, 2048)
        most = 1.0e11 / (4.0 * D * H * case["batch"] * case["q_len"])
        case["ctx"] = case["q_len"] + _log_int(rng, 1, max(1, min(14000, int(most))))
    case["q_spread"] = rng.randint(0, case["q_len"] - 1)
    case["spread"] = rng.randint(0, case["ctx"] - case["q_len"])
    if case["window"] == 0:
        case["window"] = _log_int(rng, 1, case["ctx"])
    return case


# ---------------------------------------------------------------------------- lengths, trees
def _mix(b):
    """A fixed pseudo-random number of a sequence, in [0, 2^16)."""
    return ((b * 40503 + 12345) * 2654435761 >> 12) & 0xFFFF


def _lens(case):
    """Length of each whole sequence, and its prefix; the first is the longest."""
    n = [case["len"] - (0 if b == 0 else _mix(b) * (case["spread"] + 1) >> 16) for b in range(case["batch"])]
    return n, [case["prefix"] * (0x8000 + _mix(b + 7) // 2) >> 16 for b in range(case["batch"])]


def _lengths(case):
    """(new tokens, cache length with them) of each sequence; the first has the largest of both."""
    q, kv = [], []
    for b in range(case["batch"]):
        q.append(case["q_len"] - (0 if b == 0 else _mix(b) * (case["q_spread"] + 1) >> 16))
        kv.append(case["ctx"] - (0 if b == 0 else _mix(b + 101) * (case["spread"] + 1) >> 16))
    return q, kv


def _tree(n, width):
    """Ancestors (with itself) and depth of each of n drafted tokens, `width` children to a token."""
    seen, depth = [{0}], [0]
    for i in range(1, n):
        p = (i - 1) // width
        seen.append(seen[p] | {i})
        depth.append(depth[p] + 1)
    return seen, depth


def _path(case, b, n):
    """Accepted tokens of sequence b's n drafted ones: the first, then some that stand behind the slots
    they move to, so that a second move finds what the first did."""
    m = max(1, min(case["accept"] - _mix(b + 31) * case["accept"] // (2 << 16), (n + 1) // 2))
    step = max(1, (n - m) // max(1, m - 1))
    return [0] + [m + (i - 1) * step + (_mix(b * 64 + i) * step >> 16) for i in range(1, m)]


# ---------------------------------------------------------------------------- inputs
def _randn(shape, dtype, gen, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    Hk, D = case["H_kv"], case["D"]
    st = {"case": case}
    if own:
        import exact_attention_18_gb300 as fa
        st["fa"] = fa
    if case["op"] != "keep":
        H = case["H"]
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32,
                                    device="cuda") if case["bias"] else None
        std = math.sqrt(case["gain"])  # of Q and of K
    if case["op"] in ("forward", "train"):
        lens, prefix = _lens(case)
        B, S, T = case["batch"], case["len"], sum(lens)
        q_shape = (T, H, D) if case["packed"] else (B, H, S, D)
        k_shape = (T, Hk, D) if case["packed"] else (B, Hk, S, D)
        st["q"], st["k"] = _randn(q_shape, dt, gen, std), _randn(k_shape, dt, gen, std)
        st["v"] = _randn(k_shape, dt, gen)
        if case["op"] == "train":
            st["do"] = _randn(q_shape, dt, gen)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu_host"], st["lens_host"], st["prefix_host"] = cu, lens, prefix
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st["prefix"] = torch.tensor(prefix, dtype=torch.int32, device="cuda") if case["prefix"] else None
        return st
    q_lens, kv_lens = _lengths(case)
    T, B, ps = sum(q_lens), case["batch"], case["page"]
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    pages = [-(-n // ps) for n in kv_lens]
    num_pages = sum(pages) + 3
    order = torch.randperm(num_pages, generator=gen, device="cuda")[:sum(pages)].tolist()
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    std_k = 1.0 if case["op"] == "keep" else std
    st["k_cache"] = _randn((num_pages, ps, Hk, D), dt, gen, std_k)
    st["v_cache"] = _randn((num_pages, ps, Hk, D), dt, gen)
    st["table"] = table.cuda()
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    st["q_lens_host"], st["kv_lens_host"], st["cu_host"] = q_lens, kv_lens, cu  # a scheduler knows them
    st["max_q"], st["max_k"] = max(q_lens), max(kv_lens)
    if case["op"] == "keep":
        paths = [_path(case, b, n) for b, n in enumerate(q_lens)]
        most = max(len(p) for p in paths)
        st["path"] = torch.tensor([p + [-1] * (most - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        st["path_lens"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        st["paths_host"] = paths
        return st
    st["q"] = _randn((T, H, D), dt, gen, std)
    if case["op"] == "tree":
        words = -(-st["max_q"] // 32)
        bits, pos = torch.zeros((T, words * 32), dtype=torch.int64), torch.zeros((T,), dtype=torch.int32)
        for b, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
            seen, depth = _tree(nq, case["width"])
            for i in range(nq):
                bits[cu[b] + i, sorted(seen[i])] = 1
                pos[cu[b] + i] = nk - nq + depth[i]
        weights = 2 ** torch.arange(32, dtype=torch.int64)
        word = (bits.view(T, words, 32) * weights).sum(-1)
        st["tree"] = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32).cuda()
        st["bits"] = bits.bool().cuda()
        st["pos"] = pos.cuda()
    return st


# ---------------------------------------------------------------------------- plain forms
def _modified(x, cap, slope, dist):
    """Scores from scaled products; returns (scores, derivative by the product or None)."""
    slope_of_x = None
    if cap:
        t = torch.tanh(x / cap)
        x, slope_of_x = cap * t, 1.0 - t * t
    if slope is not None:
        x = x - slope * dist
    return x, slope_of_x


def _softmax(s):
    """(weights, logsumexp) of rows; a row of -inf has weights 0."""
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m0)
    l = p.sum(-1, keepdim=True)
    return torch.where(l > 0, p / l, torch.zeros_like(p)), (m0 + torch.log(l))[..., 0]


def _hidden(c, n, prefix, device):
    i = torch.arange(n, device=device)[:, None]
    j = torch.arange(n, device=device)[None, :]
    hide = (j > i) & (j >= prefix) if c["causal"] else torch.zeros((n, n), dtype=torch.bool, device=device)
    if c["window"] >= 0:
        hide = hide | (j < i - c["window"])
        if not c["causal"]:
            hide = hide | (j > i + c["window"])
    return hide, (i - j).abs().float()


def _plain_whole(st):
    c = st["case"]
    dt, G = DTYPES[c["dtype"]], c["H"] // c["H_kv"]
    scale = 1.0 / math.sqrt(c["D"])
    train = c["op"] == "train"
    q, k, v = st["q"], st["k"], st["v"]
    o = torch.empty_like(q)
    lse = torch.empty((c["H"], q.shape[0]) if c["packed"] else q.shape[:3], dtype=torch.float32, device=q.device)
    if train:
        dq = torch.empty_like(q)
        dk, dv = (torch.zeros(k.shape, dtype=torch.float32, device=q.device) for _ in range(2))
    for b, n in enumerate(st["lens_host"]):
        hide, dist = _hidden(c, n, st["prefix_host"][b], q.device)
        rows = slice(st["cu_host"][b], st["cu_host"][b] + n)
        for h in range(c["H"]):
            at = (rows, h) if c["packed"] else (b, h)
            at_kv = (rows, h // G) if c["packed"] else (b, h // G)
            qf, kf, vf = q[at].float(), k[at_kv].float(), v[at_kv].float()
            slope = None if st["slopes"] is None else st["slopes"][h]
            s, ds_dx = _modified(torch.matmul(qf, kf.t()) * scale, c["cap"], slope, dist)
            p, l = _softmax(s.masked_fill(hide, -math.inf))
            of = torch.matmul(p, vf)
            o[at] = of.to(dt)
            lse[(h, rows) if c["packed"] else (b, h)] = l
            if train:
                do = st["do"][at].float()
                ds = p * (torch.matmul(do, vf.t()) - (do * of).sum(-1, keepdim=True))
                if ds_dx is not None:
                    ds = ds * ds_dx
                dq[at] = (torch.matmul(ds, kf) * scale).to(dt)
                dk[at_kv] += torch.matmul(ds.t(), qf) * scale
                dv[at_kv] += torch.matmul(p.t(), do)
    if train:
        return o, lse, dq, dk.to(dt), dv.to(dt)
    return o, lse


def _plain_paged(st):
    c = st["case"]
    H, Hk, D, ps, dt = c["H"], c["H_kv"], c["D"], c["page"], DTYPES[c["dtype"]]
    G, T = H // Hk, st["q"].shape[0]
    scale = 1.0 / math.sqrt(D)
    o = torch.empty((T, H, D), dtype=dt, device="cuda")
    lse = torch.empty((H, T), dtype=torch.float32, device="cuda")
    for b in range(c["batch"]):
        t0, nq, nk = st["cu_host"][b], st["q_lens_host"][b], st["kv_lens_host"][b]
        pages = st["table"][b, :-(-nk // ps)].long()
        k = st["k_cache"][pages].flatten(0, 1)[:nk]
        v = st["v_cache"][pages].flatten(0, 1)[:nk]
        j = torch.arange(nk, device="cuda")
        if c["op"] == "tree":
            i = st["pos"][t0:t0 + nq].long()
            seen = torch.ones((nq, nk), dtype=torch.bool, device="cuda")
            if c["window"] >= 0:
                seen = j[None, :] >= i[:, None] - c["window"]
            seen[:, nk - nq:] = st["bits"][t0:t0 + nq, :nq]
            j = j.clone()
            j[nk - nq:] = i
            hide = ~seen
        else:
            i = torch.arange(nk - nq, nk, device="cuda")
            hide = j[None, :] > i[:, None]
            if c["window"] >= 0:
                hide = hide | (j[None, :] < i[:, None] - c["window"])
        dist = (i[:, None] - j[None, :]).abs().float()
        for g in range(Hk):
            qg = st["q"][t0:t0 + nq, g * G:(g + 1) * G].float()
            x = torch.matmul(qg, k[:, g].float().t()) * scale
            slope = None if st["slopes"] is None else st["slopes"][g * G:(g + 1) * G, None]
            s, _ = _modified(x, c["cap"], slope, dist[:, None, :])
            p, l = _softmax(s.masked_fill(hide[:, None, :], -math.inf))
            o[t0:t0 + nq, g * G:(g + 1) * G] = torch.matmul(p, v[:, g].float()).to(dt)
            lse[g * G:(g + 1) * G, t0:t0 + nq] = l.t()
    return o, lse


def _plain_keep(st):
    ps = st["case"]["page"]
    path, lens = st["path"].long(), st["path_lens"].long()
    first = st["kv_lens"].long() - (st["cu"][1:] - st["cu"][:-1]).long()
    i = torch.arange(path.shape[1], device="cuda")[None, :]
    b, i = torch.nonzero(i < lens[:, None], as_tuple=True)
    src, dst = first[b] + path[b, i], first[b] + i
    table = st["table"].long()
    for cache in (st["k_cache"], st["v_cache"]):
        cache[table[b, dst // ps], dst % ps] = cache[table[b, src // ps], src % ps]
    return st["k_cache"], st["v_cache"]


def run(state):
    c = state["case"]
    if not own:
        return {"forward": _plain_whole, "train": _plain_whole, "paged": _plain_paged, "tree": _plain_paged,
                "keep": _plain_keep}[c["op"]](state)
    fa = state["fa"]
    if c["op"] == "keep":
        fa.paged_keep(state["k_cache"], state["v_cache"], state["table"], state["kv_lens"], state["cu"],
                      state["max_q"], state["path"], state["path_lens"])
        return state["k_cache"], state["v_cache"]
    scores = {"softcap": c["cap"] or None, "slopes": state["slopes"]}
    if c["op"] in ("paged", "tree"):
        if c["op"] == "tree":
            scores["tree"], scores["positions"] = state["tree"], state["pos"]
        return fa.forward_paged(state["q"], state["k_cache"], state["v_cache"], state["table"], state["kv_lens"],
                                state["cu"], state["max_q"], state["max_k"], causal=True,
                                window=None if c["window"] < 0 else (c["window"], 0), **scores)
    q, k, v = state["q"], state["k"], state["v"]
    scores["causal"], scores["prefix"] = c["causal"], state["prefix"]
    if c["window"] >= 0:
        scores["window"] = (c["window"], c["window"])
    packed = (state["cu"], c["len"]) if c["packed"] else ()
    o, lse = (fa.forward_varlen if c["packed"] else fa.forward)(q, k, v, *packed, **scores)
    if c["op"] == "forward":
        return o, lse
    grads = (fa.backward_varlen if c["packed"] else fa.backward)(q, k, v, o, state["do"], lse, *packed, **scores)
    return (o, lse, *grads)


# ---------------------------------------------------------------------------- work
def _pairs(c, n, prefix):
    """Visible (row, key) pairs of a whole sequence of n."""
    total = 0
    for i in range(n):
        lo = max(0, i - c["window"]) if c["window"] >= 0 else 0
        hi = max(i, prefix - 1) if c["causal"] else (min(n - 1, i + c["window"]) if c["window"] >= 0 else n - 1)
        total += max(0, min(hi, n - 1) - lo + 1)
    return total


def work(case):
    Hk, D = case["H_kv"], case["D"]
    if case["op"] == "keep":
        q_lens, _ = _lengths(case)
        rows = sum(len(_path(case, b, n)) for b, n in enumerate(q_lens))
        return {"bytes": rows * 2 * Hk * D * 2 * 2 + 4 * rows, "flops": 0}
    H = case["H"]
    if case["op"] in ("forward", "train"):
        lens, prefix = _lens(case)
        T, pairs = sum(lens), sum(_pairs(case, n, p) for n, p in zip(lens, prefix))
        train = case["op"] == "train"
        rows = (2 * H + 2 * Hk) if not train else (5 * H + 4 * Hk)  # Q, O, K, V; dO, dQ, O again, dK, dV
        return {"bytes": T * rows * D * 2 + 4 * T * H, "flops": (14 if train else 4) * D * H * pairs}
    q_lens, kv_lens = _lengths(case)
    T, pairs, keys = sum(q_lens), 0, 0
    for nq, nk in zip(q_lens, kv_lens):
        first, w = nk - nq, case["window"]
        if case["op"] == "tree":
            seen, depth = _tree(nq, case["width"])
            pairs += sum(len(s) + first - (max(0, min(first, first + d - w)) if w >= 0 else 0)
                         for s, d in zip(seen, depth))
            keys += nk - (max(0, first - w) if w >= 0 else 0)
        else:
            pairs += sum(i + 1 - (max(0, i - w) if w >= 0 else 0) for i in range(first, nk))
            keys += nk - (max(0, first - w) if w >= 0 else 0)
    return {"bytes": 2 * keys * Hk * D * 2 + 2 * T * H * D * 2 + 4 * T * H, "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------- from the definitions, in 64 bits
def _exact_scores(x, case, h, rows, keys):
    """x: scaled products [rows, keys] of head h at these positions, in 64 bits."""
    y = x if not case["cap"] else torch.tanh(x / case["cap"]) * case["cap"]
    if case["bias"]:
        slope = float(torch.tensor(2.0 ** (-8.0 * (h + 1) / case["H"]), dtype=torch.float32))
        y = y - slope * torch.abs(rows.double()[:, None] - keys.double()[None, :])
    return y


def exact(case, seed):
    st = prepare(case, seed)
    Hk, D = case["H_kv"], case["D"]
    if case["op"] == "keep":
        out = []
        for cache in (st["k_cache"], st["v_cache"]):
            old, new = cache.double(), cache.double()
            for b, path in enumerate(st["paths_host"]):
                first = st["kv_lens_host"][b] - st["q_lens_host"][b]
                slot = torch.arange(st["kv_lens_host"][b], device="cuda")
                slot = st["table"][b].long()[slot // case["page"]] * case["page"] + slot % case["page"]
                for i, t in enumerate(path):
                    new.view(-1, Hk, D)[slot[first + i]] = old.view(-1, Hk, D)[slot[first + t]]
            out.append(new)
        return tuple(out)
    H = case["H"]
    G = H // Hk
    if case["op"] in ("forward", "train"):
        if 14.0 * D * H * sum(n * n for n in st["lens_host"]) > 4.0e12:
            return None
        packed = case["packed"]
        q, k, v = (st[x].double() for x in "qkv")
        o = torch.zeros_like(q)
        lse = torch.zeros((H, q.shape[0]) if packed else q.shape[:3], dtype=torch.float64, device="cuda")
        grads = [torch.zeros_like(x) for x in (q, k, v)]
        for b, n in enumerate(st["lens_host"]):
            at = torch.arange(n, device="cuda")
            last = at.clone() if case["causal"] else torch.full_like(at, n - 1)
            if case["causal"] and st["prefix_host"][b] > 0:
                last = last.clamp_min(st["prefix_host"][b] - 1)
            first = torch.zeros_like(at)
            if case["window"] >= 0:
                first = at - case["window"]
                if not case["causal"]:
                    last = at + case["window"]
            seen = (at[None, :] >= first[:, None]) & (at[None, :] <= last[:, None])
            span = slice(st["cu_host"][b], st["cu_host"][b + 1])
            for h in range(H):
                mine = (span, h) if packed else (b, h)
                kv = (span, h // G) if packed else (b, h // G)
                x = q[mine] @ k[kv].T / math.sqrt(D)
                y = torch.where(seen, _exact_scores(x, case, h, at, at), torch.full_like(x, -math.inf))
                l = torch.logsumexp(y, -1)
                w = torch.exp(y - l[:, None])
                o[mine] = w @ v[kv]
                lse[(h, span) if packed else (b, h)] = l
                if case["op"] == "train":
                    do = st["do"][mine].double()
                    dw = do @ v[kv].T
                    dy = w * (dw - (w * dw).sum(-1, keepdim=True))
                    if case["cap"]:
                        dy = dy / torch.cosh(x / case["cap"]) ** 2
                    grads[0][mine] = dy @ k[kv] / math.sqrt(D)
                    grads[1][kv] += dy.T @ q[mine] / math.sqrt(D)
                    grads[2][kv] += w.T @ do
        return (o, lse, *grads) if case["op"] == "train" else (o, lse)
    outs, logs = [], []
    for b, (nq, nk) in enumerate(zip(st["q_lens_host"], st["kv_lens_host"])):
        key = torch.arange(nk, device="cuda")
        slot = st["table"][b].long()[key // case["page"]] * case["page"] + key % case["page"]
        span = slice(st["cu_host"][b], st["cu_host"][b + 1])
        ctx = nk - nq
        if case["op"] == "tree":
            seen_of, depth = _tree(nq, case["width"])
            row = ctx + torch.tensor(depth, device="cuda")
            seen = torch.zeros((nq, nk), dtype=torch.bool, device="cuda")
            for i in range(nq):
                seen[i, max(0, ctx + depth[i] - case["window"]) if case["window"] >= 0 else 0:ctx] = True
                seen[i, [ctx + a for a in seen_of[i]]] = True
            where = torch.cat((key[:ctx], row))
        else:
            row, where = key[ctx:], key
            seen = key[None, :] <= row[:, None]
            if case["window"] >= 0:
                seen = seen & (key[None, :] >= row[:, None] - case["window"])
        o_b = torch.empty((nq, H, D), dtype=torch.float64, device="cuda")
        l_b = torch.empty((H, nq), dtype=torch.float64, device="cuda")
        for h in range(H):
            k = st["k_cache"].view(-1, Hk, D)[slot, h // G].double()
            v = st["v_cache"].view(-1, Hk, D)[slot, h // G].double()
            y = _exact_scores((st["q"][span, h].double() @ k.T) / math.sqrt(D), case, h, row, where)
            y[~seen] = -math.inf
            l_b[h] = torch.logsumexp(y, -1)
            o_b[:, h] = torch.exp(y - l_b[h][:, None]) @ v
        outs.append(o_b)
        logs.append(l_b)
    return torch.cat(outs), torch.cat(logs, 1)
