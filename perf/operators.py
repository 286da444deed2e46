"""The operators around a paged KV cache, as a user's step calls them, next to
their plain forms in elementary torch operations.

append   qk_norm_rope_append: norm of every q and k head, position rotation,
         and the write of K and V into the cache blocks of this step's tokens.
decode   decode_masked: one query row per request over its cache blocks,
         scores capped by a tanh, with a distance bias and masks.
prefill  prefill_varlen_masked: chunks of new tokens (and decode rows) packed
         by query_start_loc, with the same scores.

Scores and masks of both attention operators, for a query at position p and a
key at position j of the same request:
    s = scale * (q . k);  s = cap * tanh(s / cap) if cap;  s -= slope_h * |p - j|
    j is visible if j < prefix_len[request] or key_start[row] <= j <= p;
a row that sees no key gives zeros.

A case's requests are "q_len:context" chunks plus `rows` requests with one new
token and lengths uniform in [lo, hi], all drawn from the case alone.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
K_SCALE, V_SCALE = 0.02, 0.017


def _case(name, op, **kw):
    base = dict(op=op, chunks="", rows=0, lo=1, hi=1, len_seed=1, heads=32, kv_heads=8, dim=128,
                block=16, e4m3=False)
    if op == "append":
        base.update(rot=128, interleaved=False, norm=True)
    else:
        base.update(cap=0.0, slopes=False, window=0, prefix=0, docs=0)
    base.update(kw)
    if name:
        base["name"] = name
    return base


def listed():
    return [
        # One request decoding alone: the latency of a single token's write.
        _case("append one token", "append", rows=1, lo=700, hi=700),
        # A decode batch of a 70B-shaped model into an e4m3 cache; half of each
        # head rotated, neighbouring pairs.
        _case("append decode batch e4m3", "append", rows=203, lo=16, hi=8192, len_seed=2, heads=64,
              e4m3=True, rot=64, interleaved=True),
        # A mixed step: one 512-token chunk and 63 decoding requests.
        _case("append mixed step", "append", chunks="512:3584", rows=63, lo=256, hi=8192, len_seed=3),
        # Long prompts, ragged, as they arrive together.
        _case("append long prompts", "append", chunks="8191:0,4097:1000,777:33,11000:0", len_seed=4),
        # The smallest batch: four short requests of a small model.
        _case("decode short", "decode", rows=4, lo=12, hi=37, len_seed=1, heads=4, kv_heads=2, dim=64,
              cap=30.0),
        # An 8B-shaped decode batch with capped scores.
        _case("decode batch capped", "decode", rows=64, lo=512, hi=4096, len_seed=2, cap=50.0),
        # Long contexts of which a 4096-token window and the first tokens are read.
        _case("decode long window", "decode", rows=8, lo=32768, hi=32768, len_seed=3, window=4096,
              prefix=64, slopes=True),
        # Eight q heads per kv head over an e4m3 cache, capped.
        _case("decode 70B e4m3 capped", "decode", rows=200, lo=16, hi=4099, len_seed=4, heads=64,
              e4m3=True, cap=30.0),
        # A mixed step with capped scores: one chunk, 63 decoding requests.
        _case("prefill mixed capped", "prefill", chunks="512:3584", rows=63, lo=256, hi=8192, len_seed=5,
              cap=50.0),
        # Prompts packed from documents that do not see each other, with a
        # distance bias; odd lengths, a few separator rows that see nothing.
        _case("prefill documents biased", "prefill", chunks="1500:0,777:0,131:259,3001:0", rows=5, lo=1,
              hi=900, len_seed=6, slopes=True, docs=300),
        # Prefix prompts of a small model: the first 576 tokens see each other.
        _case("prefill prefix e4m3", "prefill", chunks="700:0,612:0,1033:0,577:0,640:31", len_seed=7,
              heads=16, kv_heads=2, dim=64, block=32, e4m3=True, prefix=576),
        # Four long chunks with a sliding window and capped scores.
        _case("prefill long window capped", "prefill", chunks="2048:0,1024:3072,1536:6656,768:12032",
              rows=28, lo=256, hi=8192, len_seed=8, window=4096, cap=30.0),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    heads, kv_heads = rng.choice([(32, 8), (64, 8), (4, 2), (8, 8), (28, 4), (32, 2), (16, 1), (40, 8)])
    c = _case("", op, len_seed=rng.randrange(1 << 20), heads=heads, kv_heads=kv_heads,
              dim=rng.choice([64, 128, 128]), block=rng.choice([16, 16, 32, 64]), e4m3=rng.random() < 0.4)
    if op == "append":
        c.update(rot=rng.choice([c["dim"], c["dim"], c["dim"] // 2, 32]), interleaved=rng.random() < 0.4,
                 norm=rng.random() < 0.8)
    else:
        c.update(cap=rng.choice([0.0, 20.0, 30.0, 50.0]), slopes=rng.random() < 0.4,
                 prefix=rng.choice([0, 0, 4, _log_uniform(rng, 8, 1000)]))
        kind = rng.randrange(3)
        if kind == 1:
            c["window"] = _log_uniform(rng, 16, 4096)
        elif kind == 2:
            c["docs"] = _log_uniform(rng, 20, 1000)
    if op == "decode":
        c["rows"] = _log_uniform(rng, 1, 200)
        # padded K of the plain form stays below 2^31 values
        most = min(32768, (1 << 31) // (c["rows"] * kv_heads * c["dim"]))
        c["hi"] = _log_uniform(rng, 16, most)
        c["lo"] = rng.randint(1, c["hi"])
        return c
    budget = 24000 if op == "append" else 5000
    chunks = []
    for _ in range(rng.randint(0 if op == "append" else 1, 5)):
        n = _log_uniform(rng, 2, budget / 2)
        budget -= n
        chunks.append("%d:%d" % (n, rng.choice([0, rng.randint(1, 8000)])))
        if budget < 10:
            break
    c["chunks"] = ",".join(chunks)
    c["rows"] = rng.choice([0, _log_uniform(rng, 1, 63)])
    if not chunks and not c["rows"]:
        c["rows"] = 1
    c["hi"] = _log_uniform(rng, 16, 8192)
    c["lo"] = rng.randint(1, c["hi"])
    return c


def _batch(case):
    """Lengths and masks of the case's requests (numpy): seq_lens, q_lens, and
    per query row its position, key_start and request; prefix_lens."""
    rng = np.random.default_rng(case["len_seed"])
    chunks = [tuple(int(x) for x in t.split(":")) for t in case["chunks"].split(",") if t]
    rows = rng.integers(case["lo"], case["hi"], size=case["rows"], endpoint=True)
    q_lens = np.array([n for n, _ in chunks] + [1] * case["rows"], np.int64)
    seq_lens = np.array([n + c for n, c in chunks] + list(rows), np.int64)
    req = np.repeat(np.arange(len(q_lens)), q_lens)
    first = np.concatenate([[0], np.cumsum(q_lens)])
    pos = np.arange(len(req)) - first[req] + seq_lens[req] - q_lens[req]
    start = np.zeros(len(req), np.int64)
    if case.get("window"):
        start = np.maximum(start, pos - case["window"] + 1)
    if case.get("docs"):
        for r in range(len(q_lens)):
            n = int(seq_lens[r])
            cuts = np.cumsum(rng.integers(1, 2 * case["docs"], size=2 + 4 * n // case["docs"]))
            cuts = np.concatenate([[0], cuts[cuts < n]])
            p = pos[first[r]:first[r + 1]]
            start[first[r]:first[r + 1]] = cuts[np.searchsorted(cuts, p, side="right") - 1]
        start = np.where(rng.random(len(req)) < 0.01, pos + 1, start)  # separators see nothing
    prefix = np.minimum(case.get("prefix", 0), seq_lens)
    return dict(q_lens=q_lens, seq_lens=seq_lens, first=first, req=req, pos=pos, start=start, prefix=prefix)


def prepare(case, seed):
    b = _batch(case)
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    hq, hkv, d, B = case["heads"], case["kv_heads"], case["dim"], case["block"]
    S, T = len(b["q_lens"]), len(b["req"])
    need = -(-b["seq_lens"] // B)
    mb = int(need.max()) + 1
    nb = int(need.sum()) + 1 + int(need.sum()) // 8
    perm = (torch.randperm(nb - 1, generator=gen, device=dev) + 1).to(torch.int32)  # block 0: the null block
    tables = torch.zeros(S, mb, dtype=torch.int32, device=dev)
    held = torch.arange(mb, device=dev)[None, :] < torch.from_numpy(need).to(dev)[:, None]
    tables[held] = perm[: int(need.sum())]

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(device=dev, dtype=torch.int32)

    def randn(*shape, mul=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * mul).to(torch.bfloat16)

    def cache(scale):
        x = randn(nb, B, hkv, d)
        return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if case["e4m3"] else x

    s = dict(case=case, batch=b, tables=tables, seq_lens=i32(b["seq_lens"]), qsl=i32(b["first"]),
             kc=cache(K_SCALE), vc=cache(V_SCALE), pos=torch.from_numpy(b["pos"]).to(dev),
             req=torch.from_numpy(b["req"]).to(dev))
    if case["op"] == "append":
        # q, k and v of one projection's rows; k and v as views of it
        qkv = randn(T, hq + 2 * hkv, d, mul=2.0)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        rot = case["rot"]
        angle = torch.arange(int(b["seq_lens"].max()), dtype=torch.float64, device=dev)[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        for n in ("q_weight", "k_weight"):
            s[n] = 1 + 0.2 * torch.randn(d, generator=gen, device=dev) if case["norm"] else None
        s["out"] = torch.empty(T, hq, d, dtype=torch.bfloat16, device=dev)
        return s
    s["q"] = randn(T, hq, d, mul=3.0)  # trained queries give scores well beyond N(0, 1)
    s["scale"] = 1.0 / math.sqrt(d)
    s["slopes"] = (2.0 ** (-8.0 * (torch.arange(hq, device=dev) + 1) / hq)).float() if case["slopes"] else None
    masked = bool(case["window"] or case["docs"])
    s["start"] = i32(b["start"]) if masked else None
    s["prefix"] = i32(b["prefix"]) if case["prefix"] else None
    s["max_seq"], s["max_q"] = int(b["seq_lens"].max()), int(b["q_lens"].max())
    s["out"] = torch.empty_like(s["q"])
    s["ws"] = None
    if own:
        import paged_kv_cache_74_gb300 as pa
        n = pa.decode_workspace_size(S, hq, hkv, d, s["max_seq"]) if case["op"] == "decode" else \
            pa.prefill_masked_workspace_size(S, T, hq, hkv, d, s["max_seq"])
        s["ws"] = pa.new_workspace(n, dev)
    return s


# ------------------------------------------------------------ the plain forms

def _values(codes, scale):
    """A cache's values in 32 bits."""
    return codes.view(torch.float8_e4m3fn).float() * scale if codes.dtype == torch.uint8 else codes.float()


def _norm_rotate(x, weight, cos, sin, interleaved):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    h = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    head, rest = x[..., :2 * h], x[..., 2 * h:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :h], head[..., h:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, rest], -1)


def _plain_append(s):
    case, B = s["case"], s["case"]["block"]
    h = case["rot"] // 2
    cs = s["cos_sin"][s["pos"]]
    q = _norm_rotate(s["q"], s["q_weight"], cs[:, :h], cs[:, h:], case["interleaved"])
    k = _norm_rotate(s["k"], s["k_weight"], cs[:, :h], cs[:, h:], case["interleaved"])
    slot = s["tables"][s["req"], s["pos"] // B].long() * B + s["pos"] % B
    for cache, x, scale in ((s["kc"], k, K_SCALE), (s["vc"], s["v"].float(), V_SCALE)):
        if case["e4m3"]:
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache.flatten(0, 1)[slot] = x.to(cache.dtype)
    s["out"].copy_(q)
    return s["out"]


def _plain_attend(s, q, k, v, pos, start, prefix):
    """q [n, rows, hq, d] against k, v [n, keys, hkv, d] (32 bits); pos, start [n, rows], prefix [n]."""
    case = s["case"]
    n, rows, hq, d = q.shape
    keys, hkv = k.shape[1:3]
    q = q.float().view(n, rows, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    x = (q @ k.permute(0, 2, 3, 1)).view(n, hq, rows, keys) * s["scale"]
    if case["cap"]:
        x = torch.tanh(x / case["cap"]) * case["cap"]
    j = torch.arange(keys, device=q.device)
    gap = pos[:, :, None] - j
    if s["slopes"] is not None:
        x = x - s["slopes"][:, None, None] * gap.abs()[:, None]
    seen = (gap >= 0) & (j >= start[:, :, None])
    if prefix is not None:
        seen |= j < prefix[:, None, None]
    x = x.masked_fill(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total == 0, 1.0, total)
    o = w.view(n, hkv, -1, keys) @ v.permute(0, 2, 1, 3)
    return o.view(n, hq, rows, d).transpose(1, 2)


def _plain_attention(s):
    case, b, B = s["case"], s["batch"], s["case"]["block"]
    chunks = len([t for t in case["chunks"].split(",") if t])
    start = s["start"] if s["start"] is not None else torch.zeros_like(s["pos"])

    def over(requests, rows):
        """Attention of `rows` (of the packed batch) of the requests, all with the same number of rows."""
        n = requests.stop - requests.start
        keys = int(b["seq_lens"][requests].max())
        ids = s["tables"][requests, :-(-keys // B)].long()
        k = _values(s["kc"][ids], K_SCALE).flatten(1, 2)[:, :keys]
        v = _values(s["vc"][ids], V_SCALE).flatten(1, 2)[:, :keys]
        live = torch.arange(keys, device=k.device) < s["seq_lens"][requests, None]
        v = v.masked_fill(~live[..., None, None], 0)
        prefix = s["prefix"][requests] if s["prefix"] is not None else None
        o = _plain_attend(s, s["q"][rows].unflatten(0, (n, -1)), k, v, s["pos"][rows].view(n, -1),
                          start[rows].view(n, -1), prefix)
        s["out"][rows] = o.flatten(0, 1).to(torch.bfloat16)

    for r in range(chunks):  # ragged: one request at a time
        over(slice(r, r + 1), slice(int(b["first"][r]), int(b["first"][r + 1])))
    if case["rows"]:
        over(slice(chunks, chunks + case["rows"]), slice(int(b["first"][chunks]), int(b["first"][-1])))
    return s["out"]


def run(s):
    case = s["case"]
    scales = (K_SCALE, V_SCALE) if case["e4m3"] else ()
    if case["op"] == "append":
        if own:
            import paged_kv_cache_74_gb300 as pa
            call = pa.qk_norm_rope_append_fp8 if case["e4m3"] else pa.qk_norm_rope_append
            out = call(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["tables"], s["qsl"], s["seq_lens"],
                       s["cos_sin"], *scales, q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                       interleaved=case["interleaved"], out=s["out"])
        else:
            out = _plain_append(s)
        held = (s["kc"], s["vc"])
        if case["e4m3"]:
            held = tuple(c.view(torch.float8_e4m3fn) for c in held)
        return {"q": out, "key_cache": held[0], "value_cache": held[1]}
    if not own:
        return _plain_attention(s)
    import paged_kv_cache_74_gb300 as pa
    mods = dict(softcap=case["cap"], slopes=s["slopes"], key_starts=s["start"], prefix_lens=s["prefix"],
                out=s["out"], workspace=s["ws"])
    if case["op"] == "decode":
        call = pa.decode_masked_fp8 if case["e4m3"] else pa.decode_masked
        return call(s["q"], s["kc"], s["vc"], s["tables"], s["seq_lens"], s["max_seq"], s["scale"], *scales, **mods)
    call = pa.prefill_varlen_masked_fp8 if case["e4m3"] else pa.prefill_varlen_masked
    return call(s["q"], s["kc"], s["vc"], s["qsl"], s["seq_lens"], s["tables"], s["max_q"], s["max_seq"],
                s["scale"], *scales, **mods)


def work(case):
    b = _batch(case)
    T, S = len(b["req"]), len(b["q_lens"])
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    element = 1 if case["e4m3"] else 2
    if case["op"] == "append":
        rows = len(np.unique(b["pos"]))
        return {"bytes": T * d * (2 * (2 * hq + 2 * hkv) + element * 2 * hkv) + rows * case["rot"] * 4 + 4 * (2 * T + 2 * S),
                "flops": T * (hq + hkv) * (4 * d * case["norm"] + 3 * case["rot"])}
    # keys that some row of the request sees are read once; every visible (row, key) pair is computed
    start = np.maximum(b["start"], 0)
    prefix = b["prefix"][b["req"]]
    pairs = prefix + np.maximum(0, b["pos"] + 1 - np.maximum(start, prefix))
    keys = 0
    for r in range(S):
        rows = slice(b["first"][r], b["first"][r + 1])
        lo, hi = start[rows], b["pos"][rows] + 1
        hit = hi > lo
        mark = np.zeros(int(b["seq_lens"][r]) + 1, np.int64)
        np.add.at(mark, lo[hit], 1)
        np.add.at(mark, hi[hit], -1)
        mark[0] += 1
        mark[b["prefix"][r]] -= 1
        keys += int((np.cumsum(mark)[:-1] > 0).sum())
    return {"bytes": keys * hkv * d * 2 * element + T * hq * d * 4 + 4 * T * bool(case["window"] or case["docs"]) +
            4 * keys // case["block"],
            "flops": 4.0 * d * hq * float(pairs.sum())}


# ------------------------------------------------ the definitions, in 64 bits

def _slots(s, r, n):
    """Cache slots of tokens 0 .. n - 1 of request r."""
    t = torch.arange(n, device="cuda")
    return s["tables"][r].long()[t // s["case"]["block"]] * s["case"]["block"] + t % s["case"]["block"]


def _exact_head_rows(s, x, weight):
    """Norm and rotation of x [T, heads, d], as a complex rotation."""
    case = s["case"]
    x = x.double()
    if weight is not None:
        x = weight.double() * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    h = case["rot"] // 2
    turn = torch.complex(*(s["cos_sin"].double()[s["pos"]].split(h, -1)))[:, None]
    first = torch.arange(h, device=x.device) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else h)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    b, B = s["batch"], case["block"]
    if case["op"] == "append":
        slots = torch.cat([_slots(s, r, int(b["seq_lens"][r]))[-int(b["q_lens"][r]):]
                           for r in range(len(b["q_lens"]))])
        held = []
        for codes, new, scale in ((s["kc"], _exact_head_rows(s, s["k"], s["k_weight"]), K_SCALE),
                                  (s["vc"], s["v"].double(), V_SCALE)):
            if case["e4m3"]:
                new = (new / scale).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
                codes = codes.view(torch.float8_e4m3fn)
            x = codes.double()
            x.view(-1, *x.shape[2:])[slots] = new
            held.append(x)
        return {"q": _exact_head_rows(s, s["q"], s["q_weight"]), "key_cache": held[0], "value_cache": held[1]}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    pools = []
    for codes, scale in ((s["kc"], K_SCALE), (s["vc"], V_SCALE)):
        codes = codes.view(-1, *codes.shape[2:])
        pools.append((codes.view(torch.float8_e4m3fn), scale) if case["e4m3"] else (codes, 1.0))
    for r in range(len(b["q_lens"])):
        n = int(b["seq_lens"][r])
        slots = _slots(s, r, n)
        k, v = (p[slots].double() * c if not case["e4m3"] else
                p.view(torch.uint8)[slots].view(torch.float8_e4m3fn).double() * c for p, c in pools)
        j = torch.arange(n, device="cuda")
        for at in range(int(b["first"][r]), int(b["first"][r + 1]), 512):
            rows = slice(at, min(at + 512, int(b["first"][r + 1])))
            p = s["pos"][rows, None]
            seen = (j <= p) & (j >= torch.from_numpy(b["start"][rows]).cuda()[:, None])
            seen = (seen | (j < int(b["prefix"][r])))[:, None, :]
            for h in range(case["kv_heads"]):
                hs = slice(h * group, (h + 1) * group)
                e = torch.einsum("rgd,jd->rgj", s["q"][rows, hs].double(), k[:, h]) / math.sqrt(case["dim"])
                if case["cap"]:
                    e = case["cap"] * torch.tanh(e / case["cap"])
                if s["slopes"] is not None:
                    e = e - s["slopes"][hs].double()[:, None] * (p - j).abs()[:, None, :]
                e = torch.where(seen, e, -math.inf)
                weight = torch.where(seen, torch.exp(e - torch.logsumexp(e, -1, keepdim=True)), 0.0)
                out[rows, hs] = torch.einsum("rgj,jd->rgd", weight, v[:, h])
    return out
