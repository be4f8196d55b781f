"""Workloads of the prompt-side operators: rotary positions (rope), appending runs of new tokens to a cache with the rotation
applied on the way (append), and attention of a chunk of new tokens over a cache (attend).

A case is a dict of plain values. ``new`` and ``lens`` list, per sequence, how many tokens the call brings and how many rows the cache
holds (before the call for append; after it, the new ones included, for attend). ``page`` is the page size (0: dense cache).
Where ``own`` is false, ``run`` computes the plain form with elementary torch operations in 32 bits (angles in 64), rounded once.
"""
import math

import numpy as np
import torch

own = False

HALF, INTERLEAVED = 0, 1


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the queries of one decode step of 16 sequences, one layer (32 query heads): the smallest call, all latency
        dict(name="rope_decode", op="rope", layers=1, tokens=16, heads=32, d=128, layout=HALF, rot=128,
             scaling="plain", inverse=False),
        # half of a 64-wide head rotated, pairs side by side, an odd number of prompt tokens
        dict(name="rope_partial", op="rope", layers=1, tokens=4099, heads=32, d=64, layout=INTERLEAVED, rot=32,
             scaling="smooth", inverse=False),
        # un-rotating cached queries of about 10k calibration tokens, two layers
        dict(name="rope_unrotate", op="rope", layers=2, tokens=10240, heads=32, d=128, layout=HALF, rot=128,
             scaling="plain", inverse=True),
        # one decode step of 8 sequences, all 36 layers in one call, queries rotated with it
        dict(name="append_decode", op="append", layers=36, hkv=8, group=4, d=128, page=64, layout=HALF, rot=128,
             scaling="plain", new=_text([1] * 8), lens=_text([63, 64, 100, 127, 1, 0, 30, 77])),
        # drafts and short prompts of mixed lengths, small pages, part of the head rotated
        dict(name="append_ragged", op="append", layers=1, hkv=4, group=2, d=64, page=16, layout=INTERLEAVED, rot=32,
             scaling="smooth", new="1,5,700,0,129,17,64,333", lens="0,31,16,5,700,1,15,48"),
        # prompts that begin a batch of 4, one layer, positions scaled for a long context
        dict(name="append_prefill", op="append", layers=1, hkv=8, group=4, d=128, page=64, layout=HALF, rot=128,
             scaling="yarn", new="8192,3001,517,2048", lens="0,64,1000,0"),
        # one decode step of 16 sequences over a dense cache one prune interval past its budget
        dict(name="attend_decode", op="attend", layers=1, hkv=8, group=4, d=128, page=0, causal=True,
             new=_text([1] * 16), lens=_text([2176] * 16)),
        # a single token of a single long sequence: few rows, a long axis
        dict(name="attend_one_32k", op="attend", layers=1, hkv=8, group=8, d=128, page=64, causal=True,
             new="1", lens="32768"),
        # verification of 5 drafted tokens of 8 sequences, four layers in one call
        dict(name="attend_verify", op="attend", layers=4, hkv=8, group=4, d=128, page=64, causal=True,
             new=_text([5] * 8), lens="3200,3100,2053,2900,3199,2176,2500,2048"),
        # a chunk of 512 prompt tokens over a 32k cache
        dict(name="attend_chunk", op="attend", layers=1, hkv=8, group=8, d=128, page=64, causal=True,
             new="512", lens="32768"),
        # two whole prompts
        dict(name="attend_prefill", op="attend", layers=1, hkv=8, group=4, d=128, page=64, causal=True,
             new="8192,6145", lens="8192,6145"),
        # decoding and prefilling sequences in one call, narrow heads, small pages, every query sees the whole cache
        dict(name="attend_mixed", op="attend", layers=1, hkv=4, group=2, d=64, page=16, causal=False,
             new="1,1,1,1,1,1,1,1,300,77,1001,512", lens="700,1,2176,4000,129,3333,16,1500,900,77,4097,2000"),
    ]


def _text(v):
    return ",".join(str(int(x)) for x in v)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    d = rng.choice([64, 128])
    hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    turn = dict(layout=rng.choice([HALF, INTERLEAVED]), rot=rng.choice([d, d, d // 2, 3 * d // 4]),
                scaling=rng.choice(["plain", "linear", "ntk", "yarn", "smooth"]))
    if op == "rope":
        heads = hkv * group
        tokens = _log_int(rng, 1, min(20000, 20_000_000 // (heads * d)))
        return dict(op=op, layers=rng.choice([1, 1, 2, 4]), tokens=tokens, heads=heads, d=d,
                    inverse=rng.random() < 0.3, **turn)
    page = rng.choice([16, 48, 64, 64, 128, 0])
    if op == "append":
        batch = _log_int(rng, 1, 24)
        layers = rng.choice([1, 1, 2, 4])
        top = max(1, min(8192, 30_000_000 // (layers * batch * hkv * (group + 2) * d)))
        new = [rng.choice([0, 1, 1, _log_int(rng, 1, top)]) for _ in range(batch)]
        new[rng.randrange(batch)] = _log_int(rng, 1, top)
        lens = [rng.choice([0, _log_int(rng, 1, 1500)]) for _ in range(batch)]
        return dict(op=op, layers=layers, hkv=hkv, group=group, d=d, page=page, new=_text(new), lens=_text(lens), **turn)
    kind = rng.choice(["decode", "short", "chunk", "prefill", "mixed"])
    if kind == "decode":
        new = [1] * _log_int(rng, 1, 48)
        lens = [_log_int(rng, 1, 12000) for _ in new]
    elif kind == "short":
        new = [rng.randint(1, 9) for _ in range(_log_int(rng, 1, 24))]
        lens = [n + _log_int(rng, 1, 8000) for n in new]
    elif kind == "chunk":
        new = [_log_int(rng, 32, 1024)]
        lens = [new[0] + _log_int(rng, 128, 30000)]
    elif kind == "prefill":
        new = [_log_int(rng, 64, 4096) for _ in range(rng.randint(1, 3))]
        lens = list(new)
    else:
        new = [rng.choice([1, 1, _log_int(rng, 2, 800)]) for _ in range(_log_int(rng, 2, 16))]
        lens = [n + rng.choice([0, _log_int(rng, 1, 4000)]) for n in new]
    return dict(op=op, layers=1, hkv=hkv, group=group, d=d, page=page, causal=rng.random() < 0.8,
                new=_text(new), lens=_text(lens))


# ---- inputs ----------------------------------------------------------------------------------

_BASE = 1e6


def _frequencies(rot, scaling):
    """(omega fp64 [rot/2], magnitude): base^(-2f/rot), for a long context by one of the published rules
    (factor 4 past 8192 positions)."""
    w = _BASE ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot)
    factor, length = 4.0, 8192.0
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "ntk":
        return (_BASE * factor ** (rot / (rot - 2.0))) ** (-2.0 * np.arange(rot // 2, dtype=np.float64) / rot), 1.0
    if scaling == "yarn":
        def band(turns):
            return rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(_BASE))
        lo, hi = max(math.floor(band(32.0)), 0), min(math.ceil(band(1.0)), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return w * (1 - ramp) + w / factor * ramp, 0.1 * math.log(factor) + 1.0
    if scaling == "smooth":
        turns = length * w / (2 * math.pi)
        mix = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return w / factor * (1 - mix) + w * mix, 1.0
    return w, 1.0


def _normal(gen, shape, sigma):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, sigma, generator=gen).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.default_rng(seed)
    s = dict(case=case)
    L, d = case["layers"], case["d"]
    if case["op"] != "attend":
        w, s["magnitude"] = _frequencies(case["rot"], case["scaling"])
        s["omega_host"] = w
        s["omega"] = torch.from_numpy(w).cuda()
    if case["op"] == "rope":
        s["x"] = _normal(gen, (L, case["tokens"], case["heads"], d), 2.0)
        s["out"] = torch.empty_like(s["x"])
        s["pos"] = torch.from_numpy(host.integers(0, 32768, case["tokens"], dtype=np.int32)).cuda()
        return s
    new, lens = _ints(case["new"]), _ints(case["lens"])
    hkv, hq, B, T = case["hkv"], case["hkv"] * case["group"], len(new), sum(new)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s["cu"] = torch.from_numpy(cu).cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    total = [a + b for a, b in zip(new, lens)] if case["op"] == "append" else lens
    page = case["page"]
    if page:
        pages = max(1, -(-max(total) // page))
        n_pages = sum(-(-t // page) for t in total) + 1
        table = np.full((B, pages), -1, dtype=np.int32)  # -1: not allocated
        order, at = host.permutation(n_pages), 0
        for b, t in enumerate(total):
            k = -(-t // page)
            table[b, :k] = order[at:at + k]
            at += k
        s["table"] = torch.from_numpy(table).cuda()
        shape = (L, n_pages, hkv, page)
    else:
        s["table"] = None
        shape = (L, B, hkv, max(1, max(total)))
    s["K"], s["V"] = _normal(gen, shape + (d,), 0.6), _normal(gen, shape + (d,), 1.0)
    # where each token's row is: its sequence and its place among the sequence's new tokens
    seq = np.repeat(np.arange(B), new)
    place = np.arange(T) - cu[seq]
    s["seq"], s["place"] = torch.from_numpy(seq).cuda(), torch.from_numpy(place).cuda()
    if case["op"] == "append":
        s["P"] = torch.full(shape, -1, dtype=torch.int32, device="cuda")
        s["lens_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        # one projection's output: queries, keys and values of a token side by side
        qkv = _normal(gen, (L, T, hq + 2 * hkv, d), 1.0)
        s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        s["q_out"] = torch.empty((L, T, hq, d), dtype=torch.bfloat16, device="cuda")
        # a pruned cache's next position is at or past its length
        first = np.array(lens) + host.integers(0, 20000, B)
        s["pos"] = torch.from_numpy((first[seq] + place).astype(np.int32)).cuda()
    else:
        s["q"] = _normal(gen, (L, T, hq, d), 2.0)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((L, T, hq), dtype=torch.float32, device="cuda")
    return s


# ---- the plain forms -------------------------------------------------------------------------

def _turn(x, pos, omega, layout, rot, magnitude, inverse):
    """Rows x [..., T, H, d] rotated at pos [T], in fp32."""
    ang = pos.double()[:, None, None] * omega
    c, n = torch.cos(ang), torch.sin(ang)
    c, n = (c / magnitude, -n / magnitude) if inverse else (c * magnitude, n * magnitude)
    c, n, x = c.float(), n.float(), x.float()
    out = x.clone()
    if layout == HALF:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2] = a * c - b * n
        out[..., rot // 2:rot] = a * n + b * c
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2] = a * c - b * n
        out[..., 1:rot:2] = a * n + b * c
    return out


def _plain_rope(s):
    c = s["case"]
    s["out"].copy_(_turn(s["x"], s["pos"], s["omega"], c["layout"], c["rot"], s["magnitude"], c["inverse"]))
    return s["out"]


def _plain_append(s):
    c = s["case"]
    how = (s["pos"], s["omega"], c["layout"], c["rot"], s["magnitude"], False)
    slot = s["lens"].long()[s["seq"]] + s["place"]
    if c["page"]:
        at, off = s["table"].long()[s["seq"], slot // c["page"]], slot % c["page"]
    else:
        at, off = s["seq"], slot
    s["K"][:, at, :, off] = _turn(s["k"], *how).to(torch.bfloat16).transpose(0, 1)
    s["V"][:, at, :, off] = s["v"].transpose(0, 1)
    s["P"][:, at, :, off] = s["pos"][:, None, None]
    s["q_out"].copy_(_turn(s["q"], *how))
    torch.add(s["lens"], s["cu"][1:] - s["cu"][:-1], out=s["lens_out"])
    return [s["K"], s["V"], s["P"], s["lens_out"], s["q_out"]]


def _plain_attend(s):
    c = s["case"]
    new, lens = _ints(c["new"]), _ints(c["lens"])
    B, nmax, kmax, L, hkv, G, d = len(new), max(new), max(lens), c["layers"], c["hkv"], c["group"], c["d"]
    slot = torch.arange(kmax, device="cuda")
    have = slot < s["lens"][:, None]
    if c["page"]:
        at = s["table"].long()[:, slot // c["page"]].clamp_min(0)
        off = (slot % c["page"]).expand(B, kmax)
        k, v = (x[:, at, :, off].permute(2, 0, 3, 1, 4).float() for x in (s["K"], s["V"]))
    else:
        k, v = s["K"][..., :kmax, :].float(), s["V"][..., :kmax, :].float()
    v = torch.where(have[None, :, None, :, None], v, 0.0)
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(nmax, device="cuda")
    tok = (s["cu"][:-1].long()[:, None] + i).clamp_max(s["q"].shape[1] - 1)
    q = s["q"][:, tok].reshape(L, B, nmax, hkv, G, d).permute(0, 1, 3, 4, 2, 5).reshape(L, B, hkv, G * nmax, d).float()
    w = torch.matmul(q * (1.0 / math.sqrt(d)), k.transpose(-1, -2)).view(L, B, hkv, G, nmax, kmax)
    del k
    last = s["lens"].long()[:, None] - n[:, None] + i + 1 if c["causal"] else s["lens"].long()[:, None].expand(B, nmax)
    seen = have[:, None, :] & (slot < last[..., None])
    w.masked_fill_(~seen[None, :, None, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    w.sub_(m0).exp_()
    z = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(L, B, hkv, G * nmax, kmax), v).view(L, B, hkv, G, nmax, d)
    o = torch.where(z > 0, o / z, 0.0)
    lse = torch.where(z > 0, m + torch.log(z), -math.inf)
    row = (slice(None), s["seq"], slice(None), slice(None), s["place"])
    s["out"].copy_(o[row].transpose(0, 1).reshape(s["out"].shape))
    s["lse"].copy_(lse[row].transpose(0, 1).reshape(s["lse"].shape))
    return [s["out"], s["lse"]]


# ---- the framework's calls -------------------------------------------------------------------

_contexts = {}


def _context(s):
    """The context that a program keeps for its model (its shape and rotary table are loaded once)."""
    from rope_aware_key_tri_b200 import TriContext
    c = s["case"]
    hkv, G = (c["heads"], 1) if c["op"] == "rope" else (c["hkv"], c["group"])
    key = (c["layers"], hkv, G, c["d"], c.get("layout"), c.get("rot"), c.get("scaling"))
    if key not in _contexts:
        ctx = TriContext(torch.cuda.current_device())
        hq, F = hkv * G, c["d"] // 2
        ctx.calibrate_load(c["layers"], hkv, G, c["d"], _BASE, c.get("layout", HALF), np.zeros((c["layers"], hq, c["d"])),
                           np.zeros((c["layers"], hq, F)), np.zeros((c["layers"], hq, F)), [1])
        if "omega_host" in s:
            ctx.rope_load(s["omega_host"], c["layout"], magnitude=s["magnitude"])
        _contexts[key] = ctx
    return _contexts[key]


def _own(s):
    c, ctx = s["case"], _context(s)
    if c["op"] == "rope":
        return ctx.rope(s["x"], s["pos"], out=s["out"], inverse=c["inverse"])
    if c["op"] == "append":
        ctx.append_chunk(s["K"], s["V"], s["P"], s["lens"], s["k"], s["v"], s["cu"], s["pos"], lens_out=s["lens_out"],
                         block_table=s["table"], rotate=True, q=s["q"], q_out=s["q_out"])
        return [s["K"], s["V"], s["P"], s["lens_out"], s["q_out"]]
    ctx.chunk_attention(s["K"], s["V"], s["lens"], s["q"], s["cu"], out=s["out"], lse=s["lse"],
                        block_table=s["table"], causal=c["causal"])
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[state["case"]["op"]](state)


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    L, d = case["layers"], case["d"]
    if case["op"] == "rope":
        n = L * case["tokens"] * case["heads"]
        return {"bytes": 4.0 * n * d + 4.0 * case["tokens"], "flops": 3.0 * n * case["rot"]}
    new, lens = _ints(case["new"]), _ints(case["lens"])
    hkv, hq, T, B = case["hkv"], case["hkv"] * case["group"], sum(new), len(new)
    if case["op"] == "append":
        rows = L * T * (hq + 2 * hkv)
        table = 4.0 * sum(-(-(a + b) // case["page"]) - b // case["page"] for a, b in zip(new, lens)) if case["page"] else 0.0
        return {"bytes": 4.0 * rows * d + 4.0 * L * T * hkv + 4.0 * T + 12.0 * B + table,
                "flops": 3.0 * L * T * (hq + hkv) * case["rot"]}
    pairs, used = 0, 0
    for n, k in zip(new, lens):
        if case["causal"]:
            first = max(k - n + 1, 0)  # keys that the first query sees; the last sees k
            short = max(n - k, 0)      # queries that see none
            pairs += (first + k) * (n - short) // 2 if short == 0 else k * (k + 1) // 2
        else:
            pairs += n * k
        used += k if n else 0
    table = 4.0 * sum(-(-k // case["page"]) for k in lens) if case["page"] else 0.0
    return {"bytes": L * (4.0 * T * hq * d + 4.0 * T * hq + 4.0 * used * hkv * d) + 8.0 * B + table,
            "flops": 4.0 * L * hq * d * pairs}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _spun(x, pos, omega, layout, rot, magnitude, inverse):
    """Each band as a complex number, times M e^{i omega p} (or its inverse)."""
    y = x.double()
    z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) if layout == HALF else torch.view_as_complex(
        y[..., :rot].reshape(y.shape[:-1] + (rot // 2, 2)).contiguous())
    ang = (pos.double()[:, None] * omega[None, :])[:, None, :]
    e = torch.polar(torch.full_like(ang, magnitude), ang)
    z = z / e if inverse else z * e
    turned = torch.cat([z.real, z.imag], -1) if layout == HALF else torch.view_as_real(z).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _spun(s["x"], s["pos"], s["omega"], case["layout"], case["rot"], s["magnitude"], case["inverse"])
    new, lens, page = _ints(case["new"]), _ints(case["lens"]), case["page"]
    L, hkv, G, d = case["layers"], case["hkv"], case["group"], case["d"]
    ends = np.cumsum(new)
    if case["op"] == "append":
        K, V, P = s["K"].double(), s["V"].double(), s["P"].clone()
        args = (s["pos"], s["omega"], case["layout"], case["rot"], s["magnitude"], False)
        k, v = _spun(s["k"], *args), s["v"].double()
        for b in range(len(new)):
            j, done = 0, int(ends[b]) - new[b]
            while j < new[b]:  # one stretch of slots at a time: the rest of a page, or all of a dense run
                slot = lens[b] + j
                unit, off = (int(s["table"][b, slot // page]), slot % page) if page else (b, slot)
                m = min(new[b] - j, page - off) if page else new[b]
                t = slice(done + j, done + j + m)
                K[:, unit, :, off:off + m] = k[:, t].transpose(1, 2)
                V[:, unit, :, off:off + m] = v[:, t].transpose(1, 2)
                P[:, unit, :, off:off + m] = s["pos"][t]
                j += m
        total = torch.tensor([a + b for a, b in zip(new, lens)], dtype=torch.int32)
        return [K, V, P, total, _spun(s["q"], *args)]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(new, lens)):
        if n == 0 or m == 0:
            continue
        t = slice(int(ends[b]) - n, int(ends[b]))
        sees = torch.arange(n, device="cuda") + (m - n + 1) if case["causal"] else torch.full((n,), m, device="cuda")
        hidden = torch.arange(m, device="cuda")[None, :] >= sees[:, None]
        for l in range(L):
            for g in range(hkv):
                if page:
                    ids = s["table"][b, :-(-m // page)].long()
                    k, v = (x[l, ids, g].reshape(-1, d)[:m].double() for x in (s["K"], s["V"]))
                else:
                    k, v = s["K"][l, b, g, :m].double(), s["V"][l, b, g, :m].double()
                for h in range(g * G, g * G + G):
                    x = (s["q"][l, t, h].double() @ k.T) / math.sqrt(d)
                    x[hidden] = -math.inf
                    z = torch.logsumexp(x, -1)
                    p = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[:, None])
                    out[l, t, h] = p @ v
                    lse[l, t, h] = z
    return [out, lse]
