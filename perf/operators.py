"""What is measured of the cache operators: rotary positions, the append to a paged
key/value cache, and the attention of new tokens over that cache.

Each case is one call a serving or training step makes.  ``run`` computes it in
its plain form (elementary torch operations in 32 bits, angles in 64, rounded
once at the end) or, where ``own`` is true, through the library's entry points.
``exact`` gives the same outputs from the definitions in 64 bits.

Layouts: new tokens are packed, [T, heads, D], and Q, K, V are slices of one
projection [T, H + 2 H_kv, D]; the cache is [pages, page_size, H_kv, D] for K
and for V, a block table of page numbers per sequence, and a length per
sequence that counts the new tokens.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # A training step's rotation of a packed batch of 16384 tokens, 16 heads of 64.
        {"name": "rope_train_d64", "op": "rope", "dtype": "fp16", "T": 16384, "H": 16, "H_kv": 16, "D": 64, "rot": 64,
         "inter": False, "scaling": "none"},
        # The gradient of the rotation, 32 query heads on 4 K/V heads of 128.
        {"name": "rope_grad_gqa_d128", "op": "rope_bwd", "dtype": "bf16", "T": 8192, "H": 32, "H_kv": 4, "D": 128,
         "rot": 128, "inter": False, "scaling": "none"},
        # Interleaved pairs over half of the head, frequencies scaled by parts for a long context.
        {"name": "rope_inter_part_d128", "op": "rope", "dtype": "bf16", "T": 12289, "H": 32, "H_kv": 4, "D": 128,
         "rot": 64, "inter": True, "scaling": "parts"},
        # A short ragged gradient with a rotated part that no vector width divides.
        {"name": "rope_grad_odd", "op": "rope_bwd", "dtype": "fp16", "T": 1013, "H": 9, "H_kv": 3, "D": 64, "rot": 22,
         "inter": True, "scaling": "linear"},
        # One new token for each of 64 sequences: rotation and append of a decoding step.
        {"name": "append_decode_b64", "op": "append", "dtype": "bf16", "batch": 64, "q_len": 1, "q_spread": 0,
         "ctx": 2048, "spread": 1999, "H": 32, "H_kv": 4, "D": 128, "page": 16, "rot": 128, "inter": False,
         "scaling": "parts"},
        # Chunks of prompts, ragged, appended across page borders.
        {"name": "append_chunk", "op": "append", "dtype": "fp16", "batch": 6, "q_len": 2048, "q_spread": 1500,
         "ctx": 4096, "spread": 777, "H": 16, "H_kv": 2, "D": 64, "page": 64, "rot": 64, "inter": True,
         "scaling": "none"},
        # The smallest attention call: one token of one sequence.
        {"name": "decode_b1", "op": "attend", "dtype": "fp16", "batch": 1, "q_len": 1, "q_spread": 0, "ctx": 1027,
         "spread": 0, "H": 16, "H_kv": 2, "D": 64, "page": 16, "window": -1},
        # An ordinary decoding step: 32 sequences of mixed lengths.
        {"name": "decode_b32", "op": "attend", "dtype": "bf16", "batch": 32, "q_len": 1, "q_spread": 0, "ctx": 8192,
         "spread": 7000, "H": 32, "H_kv": 4, "D": 128, "page": 64, "window": -1},
        # A few long contexts: the largest read of the cache.
        {"name": "decode_long_b4", "op": "attend", "dtype": "bf16", "batch": 4, "q_len": 1, "q_spread": 0,
         "ctx": 131072, "spread": 30011, "H": 32, "H_kv": 4, "D": 128, "page": 128, "window": -1},
        # Four drafted tokens a sequence, one shared K/V head, a window over the cache.
        {"name": "draft_window_mqa", "op": "attend", "dtype": "fp16", "batch": 16, "q_len": 4, "q_spread": 3,
         "ctx": 16384, "spread": 9999, "H": 16, "H_kv": 1, "D": 64, "page": 32, "window": 4095},
        # Prompt chunks over earlier context, 8 query heads to a K/V head.
        {"name": "chunk_gqa_d128", "op": "attend", "dtype": "bf16", "batch": 2, "q_len": 2048, "q_spread": 500,
         "ctx": 16384, "spread": 4001, "H": 32, "H_kv": 4, "D": 128, "page": 64, "window": -1},
        # A mixed step: ragged chunks, some of one token, heads of 64 without grouping.
        {"name": "chunk_ragged_d64", "op": "attend", "dtype": "fp16", "batch": 8, "q_len": 1024, "q_spread": 1023,
         "ctx": 4096, "spread": 3001, "H": 16, "H_kv": 16, "D": 64, "page": 16, "window": -1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "attend", "attend", "attend"])
    D = rng.choice([16, 32, 64, 64, 128, 128])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    H = H_kv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16] if H_kv <= 4 else [1, 2, 3, 4])
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "H": H, "H_kv": H_kv, "D": D}
    if op in ("rope", "rope_bwd", "append"):
        case["rot"] = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        case["inter"] = rng.random() < 0.5
        case["scaling"] = rng.choice(["none", "linear", "base", "parts"])
    if op in ("rope", "rope_bwd"):
        most = max(2, int(4.0e7 / ((H + H_kv) * D)))
        case["T"] = _log_int(rng, 1, min(16384, most))
        return case
    case["page"] = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        case["batch"] = _log_int(rng, 1, 64)
        case["q_len"] = 1 if rng.random() < 0.4 else _log_int(rng, 1, 2048 // case["batch"] + 8)
        case["q_spread"] = rng.randint(0, case["q_len"] - 1)
        case["ctx"] = case["q_len"] + rng.randint(0, max(1, 60000 // case["batch"]))
        case["spread"] = rng.randint(0, case["ctx"] - case["q_len"])
        return case
    if rng.random() < 0.5:  # single tokens and a few drafted ones
        case["batch"] = _log_int(rng, 1, 64)
        case["q_len"] = 1 if rng.random() < 0.6 else rng.randint(2, 8)
        case["ctx"] = case["q_len"] + _log_int(rng, 1, min(131072, int(1.6e8 / (case["batch"] * H_kv * D))))
    else:                   # chunks
        case["batch"] = _log_int(rng, 1, 8)
        case["q_len"] = _log_int(rng, 9, 2048)
        case["ctx"] = case["q_len"] + _log_int(rng, 1, 14000)
        most = 4.0e11 / (4.0 * D * H * case["batch"] * case["q_len"])
        case["ctx"] = max(case["q_len"], min(case["ctx"], int(most)))
    case["q_spread"] = rng.randint(0, case["q_len"] - 1)
    case["spread"] = rng.randint(0, case["ctx"] - case["q_len"])
    case["window"] = rng.choice([-1, -1, _log_int(rng, 1, case["ctx"])])
    return case


# ---------------------------------------------------------------------------- lengths and positions
def _mix(b):
    """A fixed pseudo-random number of a sequence, in [0, 2^16)."""
    return ((b * 40503 + 12345) * 2654435761 >> 12) & 0xFFFF


def _lengths(case):
    """(new tokens, cache length with them) of each sequence; the first has the largest of both."""
    q, kv = [], []
    for b in range(case["batch"]):
        q.append(case["q_len"] - (0 if b == 0 else _mix(b) * (case["q_spread"] + 1) >> 16))
        kv.append(case["ctx"] - (0 if b == 0 else _mix(b + 101) * (case["spread"] + 1) >> 16))
    return q, kv


def _inv_freq(rot, scaling):
    """Radians per position of each pair, and the factor on cos and sin (64-bit, on the host).

    none: base^(-2i/rot); linear: that over 4; base: base * 8^(rot/(rot-2)) in base's place;
    parts: over 8 for the pairs that turn less than once in 4096 positions, unchanged for those
    that turn more than 32 times, a ramp between, and a factor 0.1 ln 8 + 1."""
    base, n = 10000.0, rot // 2
    if scaling == "base" and rot > 2:
        base = base * 8.0 ** (rot / (rot - 2))
    inv = [base ** (-2.0 * i / rot) for i in range(n)]
    mag = 1.0
    if scaling == "linear":
        inv = [f / 4.0 for f in inv]
    if scaling == "parts":
        def pair_of(turns):
            return rot * math.log(4096.0 / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
        if lo == hi:
            hi += 0.001
        for i in range(n):
            ramp = min(max((i - lo) / (hi - lo), 0.0), 1.0)
            inv[i] = inv[i] / 8.0 * ramp + inv[i] * (1.0 - ramp)
        mag = 0.1 * math.log(8.0) + 1.0
    return torch.tensor(inv, dtype=torch.float64), mag


# ---------------------------------------------------------------------------- inputs
def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    H, Hk, D = case["H"], case["H_kv"], case["D"]
    st = {"case": case}
    if own:
        import exact_attention_18_gb300 as fa
        st["fa"] = fa
    if "rot" in case:
        inv, mag = _inv_freq(case["rot"], case["scaling"])
        st["inv"], st["mag"] = inv.cuda(), mag
        if own:
            st["steps"] = fa.rope_steps(inv)
    if case["op"] in ("rope", "rope_bwd"):
        T = case["T"]
        st["x"] = _randn((T, H + 2 * Hk, D), dt, gen)  # Q, K, V (or their gradients) of one projection
        # Positions of packed sequences: each counts up from its own start, some far out.
        pos = torch.arange(T, device="cuda")
        start = torch.randint(0, 100000, (T // 1000 + 1,), generator=gen, device="cuda")
        st["pos"] = (pos % 1000 + start[pos // 1000]).to(torch.int32)
        return st
    q_lens, kv_lens = _lengths(case)
    T, B, ps = sum(q_lens), case["batch"], case["page"]
    st["x"] = _randn((T, H + 2 * Hk, D), dt, gen)
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
    st["k_cache"] = _randn((num_pages, ps, Hk, D), dt, gen)
    st["v_cache"] = _randn((num_pages, ps, Hk, D), dt, gen)
    st["table"] = table.cuda()
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    st["q_lens_host"], st["kv_lens_host"], st["cu_host"] = q_lens, kv_lens, cu  # a scheduler knows them
    st["max_q"], st["max_k"] = max(q_lens), max(kv_lens)
    if case["op"] == "attend":
        st["q"] = st["x"][:, :H].contiguous()
        del st["x"]
    return st


# ---------------------------------------------------------------------------- plain forms
def _rotate(x, pos, inv, mag, rot, inter, back, dtype):
    """Rotate the first `rot` columns of x [T, heads, D] by pos * inv, times mag; `back`: the other way."""
    ang = pos.to(torch.float64)[:, None] * inv[None, :]
    cos, sin = (torch.cos(ang) * mag).float()[:, None, :], (torch.sin(ang) * mag).float()[:, None, :]
    if back:
        sin = -sin
    y = x.float().clone()
    if inter:
        a, b = x[..., 0:rot:2].float(), x[..., 1:rot:2].float()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rot // 2
        a, b = x[..., :h].float(), x[..., h:rot].float()
        y[..., :h], y[..., h:rot] = a * cos - b * sin, b * cos + a * sin
    return y.to(dtype)


def _plain_append(st):
    c = st["case"]
    H, Hk, ps, dt = c["H"], c["H_kv"], c["page"], DTYPES[c["dtype"]]
    q, k, v = st["x"][:, :H], st["x"][:, H:H + Hk], st["x"][:, H + Hk:]
    cu, lens = st["cu"].long(), st["kv_lens"].long()
    T = q.shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.bucketize(t, cu[1:], right=True)
    pos = lens[b] - (cu[b + 1] - t)
    page = st["table"].long()[b, pos // ps]
    args = (pos, st["inv"], st["mag"], c["rot"], c["inter"], False, dt)
    st["k_cache"][page, pos % ps] = _rotate(k, *args)
    st["v_cache"][page, pos % ps] = v
    return _rotate(q, *args), st["k_cache"], st["v_cache"]


def _plain_attend(st):
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
        i = torch.arange(nk - nq, nk, device="cuda")[:, None, None]
        j = torch.arange(nk, device="cuda")[None, None, :]
        hide = j > i
        if c["window"] >= 0:
            hide = hide | (j < i - c["window"])
        for g in range(Hk):
            qg = st["q"][t0:t0 + nq, g * G:(g + 1) * G].float()
            s = torch.matmul(qg, k[:, g].float().t()) * scale
            s = s.masked_fill(hide, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            l = p.sum(-1, keepdim=True)
            o[t0:t0 + nq, g * G:(g + 1) * G] = (torch.matmul(p, v[:, g].float()) / l).to(dt)
            lse[g * G:(g + 1) * G, t0:t0 + nq] = (m + torch.log(l))[..., 0].t()
    return o, lse


def run(state):
    c = state["case"]
    H, Hk = c["H"], c["H_kv"]
    if c["op"] in ("rope", "rope_bwd"):
        q, k = state["x"][:, :H], state["x"][:, H:H + Hk]
        if own:
            f = state["fa"].rope if c["op"] == "rope" else state["fa"].rope_backward
            return f(q, k, state["pos"], state["steps"], interleaved=c["inter"], magnitude=state["mag"])
        args = (state["pos"], state["inv"], state["mag"], c["rot"], c["inter"], c["op"] == "rope_bwd",
                DTYPES[c["dtype"]])
        return _rotate(q, *args), _rotate(k, *args)
    if c["op"] == "append":
        if own:
            q, k, v = state["x"][:, :H], state["x"][:, H:H + Hk], state["x"][:, H + Hk:]
            q_rot = state["fa"].paged_append(k, v, state["k_cache"], state["v_cache"], state["table"],
                                             state["kv_lens"], state["cu"], state["max_q"], q=q,
                                             steps=state["steps"], interleaved=c["inter"], magnitude=state["mag"])
            return q_rot, state["k_cache"], state["v_cache"]
        return _plain_append(state)
    if own:
        return state["fa"].forward_paged(state["q"], state["k_cache"], state["v_cache"], state["table"],
                                         state["kv_lens"], state["cu"], state["max_q"], state["max_k"], causal=True,
                                         window=None if c["window"] < 0 else (c["window"], 0))
    return _plain_attend(state)


# ---------------------------------------------------------------------------- work
def work(case):
    H, Hk, D = case["H"], case["H_kv"], case["D"]
    if case["op"] in ("rope", "rope_bwd"):
        n = case["T"] * (H + Hk)
        return {"bytes": 2 * n * D * 2 + 4 * case["T"], "flops": 3 * n * case["rot"]}
    q_lens, kv_lens = _lengths(case)
    T = sum(q_lens)
    if case["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * Hk) * D * 2 + 8 * case["batch"], "flops": 3 * T * (H + Hk) * case["rot"]}
    pairs = keys = 0
    for nq, nk in zip(q_lens, kv_lens):
        w = nk if case["window"] < 0 else case["window"] + 1
        first = nk - nq
        if w >= nk:
            pairs += nq * (first + 1 + nk) // 2
            keys += nk
        else:
            pairs += sum(min(i + 1, w) for i in range(first, nk))
            keys += nk - max(0, first + 1 - w)
    return {"bytes": 2 * keys * Hk * D * 2 + 2 * T * H * D * 2 + 4 * T * H, "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------- from the definitions, in 64 bits
def _turned(x, angle, mag, rot, inter):
    """Pair (a, b) as the complex number a + ib, times mag * e^{i angle}; columns past rot unchanged."""
    z = x.double()
    if inter:
        w = torch.view_as_complex(z[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous())
    else:
        w = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:rot].contiguous())
    w = w * torch.polar(torch.full_like(angle, mag), angle)[:, None, :]
    if inter:
        head = torch.view_as_real(w).flatten(-2)
    else:
        head = torch.cat((w.real, w.imag), -1)
    return torch.cat((head, z[..., rot:]), -1)


def exact(case, seed):
    st = prepare(case, seed)
    H, Hk, D = case["H"], case["H_kv"], case["D"]
    if case["op"] in ("rope", "rope_bwd"):
        angle = torch.outer(st["pos"].double(), st["inv"]) * (1.0 if case["op"] == "rope" else -1.0)
        return tuple(_turned(x, angle, st["mag"], case["rot"], case["inter"])
                     for x in (st["x"][:, :H], st["x"][:, H:H + Hk]))
    ps = case["page"]
    if case["op"] == "append":
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        spans = [torch.arange(nk - nq, nk, device="cuda") for nq, nk in zip(st["q_lens_host"], st["kv_lens_host"])]
        angle = torch.outer(torch.cat(spans).double(), st["inv"])
        q, k = (_turned(x, angle, st["mag"], case["rot"], case["inter"])
                for x in (st["x"][:, :H], st["x"][:, H:H + Hk]))
        v = st["x"][:, H + Hk:].double()
        for b, at in enumerate(spans):
            rows = slice(st["cu_host"][b], st["cu_host"][b + 1])
            slot = st["table"][b].long()[at // ps] * ps + at % ps
            kc.view(-1, Hk, D)[slot] = k[rows]
            vc.view(-1, Hk, D)[slot] = v[rows]
        return q, kc, vc
    outs, logs = [], []
    for b, (nq, nk) in enumerate(zip(st["q_lens_host"], st["kv_lens_host"])):
        key = torch.arange(nk, device="cuda")
        slot = st["table"][b].long()[key // ps] * ps + key % ps
        row = torch.arange(nk - nq, nk, device="cuda")[:, None]
        seen = key[None, :] <= row
        if case["window"] >= 0:
            seen = seen & (key[None, :] >= row - case["window"])
        o_b = torch.empty((nq, H, D), dtype=torch.float64, device="cuda")
        l_b = torch.empty((H, nq), dtype=torch.float64, device="cuda")
        for h in range(H):
            g = h // (H // Hk)
            k = st["k_cache"].view(-1, Hk, D)[slot, g].double()
            v = st["v_cache"].view(-1, Hk, D)[slot, g].double()
            s = (st["q"][st["cu_host"][b]:st["cu_host"][b + 1], h].double() @ k.T) / math.sqrt(D)
            s[~seen] = -math.inf
            l_b[h] = torch.logsumexp(s, -1)
            o_b[:, h] = torch.exp(s - l_b[h][:, None]) @ v
        outs.append(o_b)
        logs.append(l_b)
    return torch.cat(outs), torch.cat(logs, 1)
