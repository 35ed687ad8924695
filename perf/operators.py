"""The paged factor cache: its cases, its operators in plain torch, and the calls a user makes.

Four operators work on one cache whose slots lie in pages of a pool, found through a page
table: writing new tokens' factor records (as bf16, or quantised to e4m3 with a power-of-two
scale per token and factor part), reading records back, attention of a ragged chunk of new
tokens, and attention of one token per sequence, both with an optional sliding window beside
the first tokens that stay visible.

Layout of a pool plane (E elements a record, P slots a page):
  bf16   [n_pages][P / 8][E][8]         element-major, token-minor in groups of 8 slots
  e4m3   [n_pages][P / 16][E + 2][16]   groups of 16 slots, slot t of a group at byte
         2 (t % 8) + t / 8 of a row; rows 0 .. E - 1 hold the codes, row E the exponent byte
         (E8M0) of the token's A factors, row E + 1 that of its B factors
A record is [A_0 .. A_{R-1} | B_0 .. B_{R-1}], A_r of h1 x d1 and B_r of h2 x d2 values; a key is
(1/R) sum_r A_r (x) B_r over h1 h2 heads of d1 d2 features, a value likewise.
"""
import math
import random

import torch

own = False

#: Head splits this repository's workloads use: (h1, h2, d1, d2, R).
SPLITS = {
    "kpa_4x8_8x16_r2": (4, 8, 8, 16, 2),
    "kpa_4x8_8x16_r4": (4, 8, 8, 16, 4),
    "kpa_4x4_8x16_r2": (4, 4, 8, 16, 2),
    "kpa_4x4_8x16_r4": (4, 4, 8, 16, 4),
    "kpa_4x4_8x8_r2": (4, 4, 8, 8, 2),
    "kpa_2x8_8x8_r2": (2, 8, 8, 8, 2),
    "tpa_16_64_r2": (16, 1, 1, 64, 2),
    "tpa_32_64_r1": (32, 1, 1, 64, 1),
    "tpa_16_128_r2": (16, 1, 1, 128, 2),
}
BASE = 10000.0


def _case(name, op, split, fmt, page, batch, lo, hi, new_lo, new_hi, window, sinks, mix):
    """lo .. hi: cached tokens of a sequence before the call (for a decode: its whole length);
    new_lo .. new_hi: its new tokens; mix: seed of those lengths."""
    c = {"op": op, "split": split, "format": fmt, "page": page, "batch": batch, "lo": lo, "hi": hi,
         "new_lo": new_lo, "new_hi": new_hi, "window": window, "sinks": sinks, "mix": mix}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decoding step of a server writes one token for each of 48 running sequences
        _case("append_step_e4m3", "append", "kpa_4x8_8x16_r2", "e4m3", 64, 48, 0, 8192, 1, 1, 0, 0, 1),
        # ragged prompt chunks into a bf16 cache of small pages
        _case("append_ragged_bf16", "append", "tpa_16_64_r2", "bf16", 16, 5, 0, 1000, 1, 777, 0, 0, 2),
        # whole prompts quantised as they are written: 8 x 2048 tokens
        _case("append_prompt_e4m3", "append", "kpa_4x4_8x16_r2", "e4m3", 128, 8, 0, 0, 2048, 2048, 0, 0, 3),
        # a few sequences' last tokens read back (moving a request, checking a cache)
        _case("read_part_e4m3", "read", "kpa_4x4_8x8_r2", "e4m3", 32, 3, 5, 3000, 50, 401, 0, 0, 4),
        # whole prompts read back from 8 bits
        _case("read_prompt_e4m3", "read", "tpa_16_128_r2", "e4m3", 64, 8, 0, 0, 2048, 2048, 0, 0, 5),
        # decoding a small batch over 4096 tokens each, small bf16 pages: latency counts
        _case("decode_step_bf16", "decode", "tpa_16_64_r2", "bf16", 16, 8, 4096, 4096, 0, 0, 0, 0, 6),
        # decoding a ragged batch at rank 4
        _case("decode_ragged_bf16", "decode", "kpa_4x8_8x16_r4", "bf16", 64, 32, 1024, 8192, 0, 0, 0, 0, 7),
        # one very long context in 8 bits
        _case("decode_long_e4m3", "decode", "kpa_4x8_8x16_r2", "e4m3", 128, 1, 524288, 524288, 0, 0, 0, 0, 8),
        # a large batch with a window of 4096 tokens and four sinks
        _case("decode_window_e4m3", "decode", "tpa_32_64_r1", "e4m3", 32, 64, 1500, 40000, 0, 0, 4096, 4, 9),
        # prompts in one chunk: 8 x 2048 tokens, causal
        _case("prefill_prompt_bf16", "prefill", "kpa_4x4_8x16_r2", "bf16", 128, 8, 0, 0, 2048, 2048, 0, 0, 10),
        # one chunk of a long prompt over what is cached already
        _case("prefill_chunk_e4m3", "prefill", "kpa_4x4_8x16_r2", "e4m3", 64, 1, 30011, 30011, 257, 257, 0, 0, 11),
        # a mixed step: single tokens and chunks of several requests, with a window and sinks
        _case("prefill_window_bf16", "prefill", "tpa_16_128_r2", "bf16", 16, 12, 0, 6000, 1, 400, 1024, 4, 12),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "prefill"])
    split = rng.choice(sorted(SPLITS))
    fmt = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    mix = rng.randrange(1 << 30)
    window, sinks = rng.choice([(0, 0), (0, 0), (_spread(rng, 16, 4096), rng.randrange(0, 20))])
    if op in ("append", "read"):
        batch = _spread(rng, 1, 64)
        most = max(1, 16384 // batch)
        new = _spread(rng, 1, most)
        return _case(None, op, split, fmt, page, batch, 0, _spread(rng, 1, 8192), max(1, new // 3), new, 0, 0, mix)
    if op == "decode":
        batch = _spread(rng, 1, 64)
        hi = _spread(rng, 1, min(400000, 400000 // batch))
        return _case(None, op, split, fmt, page, batch, rng.choice([0, hi // 2, hi]), hi, 0, 0, window, sinks, mix)
    batch = _spread(rng, 1, 8)
    new = _spread(rng, 1, 2048 if batch <= 4 else 1024)
    past = _spread(rng, 1, max(64, min(30000, 12000000 // (new * batch))))
    return _case(None, op, split, fmt, page, batch, rng.choice([0, past]), past, max(1, new // 4), new, window, sinks, mix)


def _lengths(case):
    """(cached tokens before the call, new tokens) of each sequence."""
    rng = random.Random(case["mix"])
    past = [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return past, new


def _visible(p, window, sinks):
    """Slots that the query at position p sees."""
    if not window or p + 1 <= window + sinks:
        return p + 1
    return window + sinks


def work(case):
    h1, h2, d1, d2, R = SPLITS[case["split"]]
    E, h, dh = R * (h1 * d1 + h2 * d2), h1 * h2, d1 * d2
    record = 2 * (E * 2 if case["format"] == "bf16" else E + 2)
    past, new = _lengths(case)
    w, s = case["window"], case["sinks"]
    if case["op"] in ("append", "read"):
        return {"bytes": sum(new) * (record + 4 * E), "flops": 0}
    if case["op"] == "decode":
        seen = sum(_visible(n - 1, w, s) if n else 0 for n in past)
        return {"bytes": seen * record + case["batch"] * h * dh * 4, "flops": 2 * seen * R * h * (2 * dh + 2 * d1)}
    pairs = sum(_visible(p + t, w, s) for p, n in zip(past, new) for t in range(n))
    slots = sum(min(p + n, n + w - 1 + s if w else p + n) for p, n in zip(past, new))
    return {"bytes": slots * record + sum(new) * h * dh * 4, "flops": 4 * pairs * h * dh + 4 * slots * R * h * dh}


def _byte_of_token():
    return [2 * (t % 8) + t // 8 for t in range(16)]


def _fill(gen, n_pages, page, E, a, fmt):
    """A pool plane of random records, as an earlier part of the program left it."""
    if fmt == "bf16":
        x = torch.randn(n_pages * page * E, device="cuda", generator=gen).mul_(2 ** -0.5)
        return x.to(torch.bfloat16)
    x = torch.randn(n_pages, page // 16, E, 16, device="cuda", generator=gen).mul_(2 ** -0.5)
    pool = torch.empty(n_pages, page // 16, E + 2, 16, device="cuda", dtype=torch.uint8)
    for i, part in enumerate((x[:, :, :a], x[:, :, a:])):
        e = torch.ceil(torch.log2(part.abs().amax(2, keepdim=True) / 448))
        lo = 0 if i == 0 else a
        pool[:, :, lo:lo + part.shape[2]] = (part * torch.exp2(-e)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pool[:, :, E + i] = (e[:, :, 0] + 127).to(torch.uint8)
    return pool.view(-1)


def prepare(case, seed):
    h1, h2, d1, d2, R = SPLITS[case["split"]]
    E, a, P, B = R * (h1 * d1 + h2 * d2), R * h1 * d1, case["page"], case["batch"]
    gen = torch.Generator("cuda").manual_seed(seed)
    past, new = _lengths(case)
    total = [p + n for p, n in zip(past, new)]
    cols = max(1, -(-max(total) // P))
    need = [-(-t // P) for t in total]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32).cpu()
    table = torch.full((B, cols), -1, dtype=torch.int32)       # pages a sequence does not have: -1
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    i32 = {"dtype": torch.int32, "device": "cuda"}
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st = {"case": dict(case), "n_pages": n_pages, "max_len": max(total), "max_new": max(new), "n_rows": cu[-1],
          "table": table.cuda(), "cu_rows": torch.tensor(cu, **i32), "start": torch.tensor(past, **i32),
          "seq_len": torch.tensor(past, **i32), "scale": 1.0 / math.sqrt(d1 * d2)}
    if case["op"] == "append":
        size = n_pages * P * E if case["format"] == "bf16" else n_pages * P * (E + 2)
        for k in ("kpool", "vpool"):
            st[k] = torch.zeros(size, device="cuda", dtype=torch.bfloat16 if case["format"] == "bf16" else torch.uint8)
    else:
        for k in ("kpool", "vpool"):
            st[k] = _fill(gen, n_pages, P, E, a, case["format"])
    n = cu[-1]
    if case["op"] == "append":
        for k in ("kf", "vf"):
            st[k] = torch.randn(n, E, device="cuda", generator=gen).mul_(2 ** -0.5).to(torch.bfloat16)
    elif case["op"] == "read":
        for k in ("kf", "vf"):
            st[k] = torch.empty(n, E, device="cuda", dtype=torch.bfloat16)
    else:
        rows = B if case["op"] == "decode" else n
        st["q"] = torch.randn(rows, h1 * h2, d1 * d2, device="cuda", generator=gen).mul_(0.3).to(torch.bfloat16)
        st["out"] = torch.empty_like(st["q"])
    return st


# ------------------------------------------------------------------ the framework's calls
def _own_handle(st):
    """What a user's program makes once beside its pool: the descriptors and the workspace."""
    import factorised_kv_attention_b200 as kpa
    from workloads import Shape
    c = st["case"]
    h1, h2, d1, d2, R = SPLITS[c["split"]]
    cfg = kpa.make_config(Shape(h1=h1, h2=h2, d1=d1, d2=d2, r_k=R, r_v=R, rope_base=BASE), "bf16")
    pages = kpa.make_pages(c["page"], st["n_pages"], st["table"].shape[1], c["format"])
    size = 0
    if c["op"] == "decode":
        size = kpa.kpa_paged_decode_workspace_size(cfg, pages, c["batch"], st["max_len"], c["window"], c["sinks"])
    elif c["op"] == "prefill":
        size = kpa.kpa_paged_prefill_workspace_size(cfg, pages, c["batch"], st["n_rows"], st["max_len"], c["window"], c["sinks"])
    st["own"] = (kpa, cfg, pages, torch.zeros(max(256, size), dtype=torch.uint8, device="cuda"))
    return st["own"]


def _own_run(st):
    kpa, cfg, pages, ws = st.get("own") or _own_handle(st)
    c = st["case"]
    if c["op"] == "append":
        kpa.kpa_paged_append_factors(cfg, pages, c["batch"], st["n_rows"], st["kf"], st["vf"], st["cu_rows"], st["start"],
                                     st["table"], st["kpool"], st["vpool"])
    elif c["op"] == "read":
        kpa.kpa_paged_read_factors(cfg, pages, c["batch"], st["n_rows"], st["cu_rows"], st["start"], st["table"],
                                   st["kpool"], st["vpool"], st["kf"], st["vf"])
    elif c["op"] == "decode":
        kpa.kpa_paged_decode(cfg, pages, c["batch"], st["q"], st["seq_len"], st["table"], st["kpool"], st["vpool"],
                             st["max_len"], c["window"], c["sinks"], st["scale"], st["out"], ws)
    else:
        kpa.kpa_paged_prefill(cfg, pages, c["batch"], st["n_rows"], st["q"], st["cu_rows"], st["start"], st["table"],
                              st["kpool"], st["vpool"], st["max_len"], c["window"], c["sinks"], st["scale"], st["out"], ws)


# ------------------------------------------------------------------ the plain forms
def _plane(st, pool):
    """A pool plane as [n_pages][groups of a page][rows][slots of a group]."""
    c = st["case"]
    h1, h2, d1, d2, R = SPLITS[c["split"]]
    E = R * (h1 * d1 + h2 * d2)
    if c["format"] == "bf16":
        return pool.view(st["n_pages"], c["page"] // 8, E, 8)
    return pool.view(st["n_pages"], c["page"] // 16, E + 2, 16)


def _values(st, x):
    """Records [..., rows of a group][slots in token order] as values [..., slots][E]."""
    if st["case"]["format"] == "bf16":
        return x.float().transpose(-1, -2)
    h1, h2, d1, d2, R = SPLITS[st["case"]["split"]]
    a, E = R * h1 * d1, R * (h1 * d1 + h2 * d2)
    scale = torch.exp2(x[..., E:, :].float() - 127)
    code = x[..., :E, :].view(torch.float8_e4m3fn).float()
    code = torch.cat([code[..., :a, :] * scale[..., :1, :], code[..., a:, :] * scale[..., 1:, :]], -2)
    return code.transpose(-1, -2)


def _cached(st, pool):
    """[batch][slots of the table's pages][E] values of every sequence."""
    x = _plane(st, pool)[st["table"].clamp(min=0).long()]          # B, cols, groups, rows, slots
    if st["case"]["format"] == "e4m3":
        x = x[..., torch.tensor(_byte_of_token(), device=x.device)]
    x = _values(st, x)
    return x.reshape(x.shape[0], -1, x.shape[-1])


def _factors(st, pool):
    """A [batch][slots][R][h1][d1] and B [batch][slots][R][h2][d2] of one plane."""
    h1, h2, d1, d2, R = SPLITS[st["case"]["split"]]
    x = _cached(st, pool)
    return x[..., :R * h1 * d1].unflatten(-1, (R, h1, d1)), x[..., R * h1 * d1:].unflatten(-1, (R, h2, d2))


def _rows(st):
    """Sequence and position of each row, and where its slot lies: page, slot of the page."""
    r = torch.arange(st["n_rows"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["cu_rows"][1:].contiguous(), r, right=True)
    pos = (st["start"][b] + r - st["cu_rows"][b]).long()
    return b, pos, st["table"][b, pos // st["case"]["page"]].long(), pos % st["case"]["page"]


def _seen(pos, slots, case):
    """Whether the query at pos sees each slot."""
    s = torch.arange(slots, device="cuda")
    p = pos[..., None]
    see = s <= p
    return see & ((p - s < case["window"]) | (s < case["sinks"])) if case["window"] else see


def _plain_append(st):
    c = st["case"]
    h1, h2, d1, d2, R = SPLITS[c["split"]]
    a, E = R * h1 * d1, R * (h1 * d1 + h2 * d2)
    b, pos, page, slot = _rows(st)
    angle = pos.double()[:, None] * BASE ** (-torch.arange(0, d2, 2, device="cuda", dtype=torch.float64) / d2)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = st["kf"][:, a:].float().view(-1, R * h2, d2 // 2, 2)
    turned = torch.stack([x[..., 0] * cos - x[..., 1] * sin, x[..., 0] * sin + x[..., 1] * cos], -1).flatten(1)
    k, v = torch.cat([st["kf"][:, :a].float(), turned], 1), st["vf"].float()
    if c["format"] == "bf16":
        _plane(st, st["kpool"])[page, slot // 8, :, slot % 8] = k.to(torch.bfloat16)
        _plane(st, st["vpool"])[page, slot // 8, :, slot % 8] = v.to(torch.bfloat16)
        return
    byte = 2 * (slot % 8) + slot % 16 // 8
    _plane(st, st["kpool"])[page, slot // 16, :, byte] = _quantised(k, a)
    _plane(st, st["vpool"])[page, slot // 16, :, byte] = _quantised(v, a)


def _quantised(x, a):
    """The E + 2 bytes of each record."""
    ea, eb = _exponent(x[:, :a]), _exponent(x[:, a:])
    y = torch.cat([x[:, :a] * torch.exp2(-ea), x[:, a:] * torch.exp2(-eb)], 1)
    y = torch.where(y.isfinite(), y.clamp(-448, 448), math.nan).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([y, (ea + 127).to(torch.uint8), (eb + 127).to(torch.uint8)], 1)


def _exponent(x):
    """The smallest whole e of -64 .. 63 with 448 * 2^e no less than every finite value."""
    m, e = torch.frexp(torch.where(x.isfinite(), x.abs(), 0.0).amax(1, keepdim=True))     # m in [1/2, 1)
    return torch.where(m == 0, -64.0, (e - 9 + (m > 0.875)).float()).clamp(-64, 63)


def _plain_read(st):
    b, pos, page, slot = _rows(st)
    c = st["case"]
    if c["format"] == "bf16":
        st["kf"].copy_(_plane(st, st["kpool"])[page, slot // 8, :, slot % 8])
        st["vf"].copy_(_plane(st, st["vpool"])[page, slot // 8, :, slot % 8])
        return
    byte = 2 * (slot % 8) + slot % 16 // 8
    st["kf"].copy_(_values(st, _plane(st, st["kpool"])[page, slot // 16, :, byte][..., None])[:, 0])
    st["vf"].copy_(_values(st, _plane(st, st["vpool"])[page, slot // 16, :, byte][..., None])[:, 0])


def _softmax(score, see):
    """Softmax over the last axis of what is seen; zeros where nothing is."""
    score = torch.where(see, score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top)
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_decode(st):
    c = st["case"]
    h1, h2, d1, d2, R = SPLITS[c["split"]]
    A, Bf = _factors(st, st["kpool"])
    q = st["q"].float().view(-1, h1, h2, d1, d2)
    T = torch.einsum("bxyij,blryj->blrxyi", q, Bf)
    score = torch.einsum("blrxyi,blrxi->bxyl", T, A) * (st["scale"] / R)
    del T, A, Bf
    pos = st["seq_len"].long() - 1
    p = _softmax(score, _seen(pos, score.shape[-1], c)[:, None, None])
    A, Bf = _factors(st, st["vpool"])
    W = torch.einsum("bxyl,blrxi->blrxyi", p, A)
    O = torch.einsum("blrxyi,blryj->bxyij", W, Bf) / R
    st["out"].copy_(O.reshape(st["out"].shape))


def _dense(st, pool):
    """[batch][heads][slots][d_h] keys or values."""
    A, Bf = _factors(st, pool)
    x = torch.einsum("blrxi,blryj->bxylij", A, Bf) / A.shape[2]
    return x.flatten(4, 5).flatten(1, 2)


def _plain_prefill(st):
    c = st["case"]
    n = torch.arange(st["max_new"], device="cuda")
    row = (st["cu_rows"][:-1, None].long() + n).clamp(max=st["n_rows"] - 1)     # padded to the longest chunk
    q = st["q"][row].float().transpose(1, 2)                                    # B, h, n, dh
    score = q @ _dense(st, st["kpool"]).transpose(-1, -2) * st["scale"]
    see = _seen(st["start"][:, None].long() + n, score.shape[-1], c)
    O = _softmax(score, see[:, None]) @ _dense(st, st["vpool"])                 # B, h, n, dh
    b, pos, _, _ = _rows(st)
    st["out"].copy_(O.transpose(1, 2)[b, pos - st["start"][b].long()])


def _outputs(st):
    op = st["case"]["op"]
    if op == "read":
        return {"k": st["kf"], "v": st["vf"]}
    if op != "append":
        return st["out"]
    k, v = _plane(st, st["kpool"]), _plane(st, st["vpool"])
    if st["case"]["format"] == "bf16":
        return {"k": k, "v": v}
    return {"k": k[:, :, :-2].view(torch.float8_e4m3fn), "v": v[:, :, :-2].view(torch.float8_e4m3fn),
            "k_scale": k[:, :, -2:].view(torch.float8_e8m0fnu), "v_scale": v[:, :, -2:].view(torch.float8_e8m0fnu)}


def run(state):
    if own:
        _own_run(state)
    else:
        {"append": _plain_append, "read": _plain_read, "decode": _plain_decode, "prefill": _plain_prefill}[state["case"]["op"]](state)
    return _outputs(state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_records(st, pool, b, upto, device="cuda"):
    """Records 0 .. upto - 1 of sequence b in 64 bits, slot by slot of the layout."""
    c = st["case"]
    h1, h2, d1, d2, R = SPLITS[c["split"]]
    E, a, P = R * (h1 * d1 + h2 * d2), R * h1 * d1, c["page"]
    s = torch.arange(upto, device=device)
    page = st["table"][b].long()[s // P]
    e = torch.arange(E, device=device)
    if c["format"] == "bf16":
        at = ((page * P + s % P) // 8)[:, None] * (8 * E) + e * 8 + (s % 8)[:, None]
        return pool[at].double()
    group = ((page * P + s % P) // 16)[:, None] * (16 * (E + 2))
    byte = (2 * (s % 8) + s % 16 // 8)[:, None]
    code = pool[group + e * 16 + byte].view(torch.float8_e4m3fn).double()
    power = pool[group + torch.where(e < a, E, E + 1) * 16 + byte].double() - 127
    return code * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=device), power)


def _exact_attention(st):
    c = st["case"]
    h1, h2, d1, d2, R = SPLITS[c["split"]]
    a, cu = R * h1 * d1, st["cu_rows"].tolist()
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        if c["op"] == "decode":
            n, first, last = int(st["seq_len"][b]), b, b + 1
            if n == 0:
                continue
            pos = torch.tensor([n - 1], device="cuda")
        else:
            first, last = cu[b], cu[b + 1]
            n = int(st["start"][b]) + last - first
            pos = torch.arange(n - (last - first), n, device="cuda")
        k, v = _exact_records(st, st["kpool"], b, n), _exact_records(st, st["vpool"], b, n)
        s = torch.arange(n, device="cuda")
        hidden = s[None] > pos[:, None]
        if c["window"]:
            hidden |= (pos[:, None] - s[None] >= c["window"]) & (s[None] >= c["sinks"])
        for h in range(h1 * h2):
            x, y = h // h2, h % h2
            K = sum(k[:, (r * h1 + x) * d1:(r * h1 + x + 1) * d1, None] * k[:, None, a + (r * h2 + y) * d2:a + (r * h2 + y + 1) * d2]
                    for r in range(R)).flatten(1) / R
            V = sum(v[:, (r * h1 + x) * d1:(r * h1 + x + 1) * d1, None] * v[:, None, a + (r * h2 + y) * d2:a + (r * h2 + y + 1) * d2]
                    for r in range(R)).flatten(1) / R
            z = (st["q"][first:last, h].double() @ K.T) * (1.0 / math.sqrt(d1 * d2))
            out[first:last, h] = torch.softmax(z.masked_fill(hidden, -math.inf), 1) @ V
    return out


def _exact_append(st):
    c = st["case"]
    h1, h2, d1, d2, R = SPLITS[c["split"]]
    E, a, P = R * (h1 * d1 + h2 * d2), R * h1 * d1, c["page"]
    cu, start = st["cu_rows"].tolist(), st["start"].tolist()
    bf16 = c["format"] == "bf16"
    k, v = (torch.zeros(_plane(st, st[p]).shape, dtype=torch.float64, device="cuda") for p in ("kpool", "vpool"))
    for b in range(c["batch"]):
        pos = torch.arange(start[b], start[b] + cu[b + 1] - cu[b], device="cuda")
        page, slot = st["table"][b].long()[pos // P], pos % P
        theta = torch.tensor([BASE ** (-2.0 * m / d2) for m in range(d2 // 2)], dtype=torch.float64, device="cuda")
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * theta)[:, None]
        kx = st["kf"][cu[b]:cu[b + 1]].double()
        kx[:, a:] = torch.view_as_real(torch.view_as_complex(kx[:, a:].reshape(-1, R * h2, d2 // 2, 2).contiguous()) * z).flatten(1)
        for plane, x in ((k, kx), (v, st["vf"][cu[b]:cu[b + 1]].double())):
            if bf16:
                plane[page, slot // 8, :, slot % 8] = x
                continue
            e = [torch.ceil(torch.log2(part.abs().amax(1, keepdim=True) / 448)).clamp(-64, 63) for part in (x[:, :a], x[:, a:])]
            y = torch.cat([x[:, :a] / 2 ** e[0], x[:, a:] / 2 ** e[1], 2 ** e[0], 2 ** e[1]], 1)
            plane[page, slot // 16, :, 2 * (slot % 8) + slot % 16 // 8] = y
    if bf16:
        return {"k": k, "v": v}
    # the codes' values before their rounding; the scales of slots that the call does not write are no computed numbers
    return {"k": k[:, :, :-2], "v": v[:, :, :-2], "k_scale": None, "v_scale": None}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] in ("decode", "prefill"):
        return _exact_attention(st)
    cu, start = st["cu_rows"].tolist(), st["start"].tolist()
    found = {}
    for name, pool in (("k", st["kpool"]), ("v", st["vpool"])):
        rows = [_exact_records(st, pool, b, start[b] + cu[b + 1] - cu[b])[start[b]:] for b in range(case["batch"])]
        found[name] = torch.cat(rows)
    return found
