"""The operators of a speculative step over a paged KV cache, as a user's step
calls them, next to their plain forms in elementary torch operations.

step    plan_step: from the requests' lengths, the cache blocks of the new tokens
        (taken off a stack of free ones and entered in the block tables), the
        step's row offsets, lengths, slots and positions, and the ancestor masks
        of drafted token trees; then release_blocks: the blocks past the kept
        lengths go back on the stack, as after a step that kept nothing.
attend  tree_attention: the drafted tokens of each request over its cache; a row
        sees the whole context and, of the request's new tokens, those its mask
        names.
commit  commit_tokens: K and V of the accepted drafted tokens move to the slots
        behind the context, in every layer.

A case's requests are "new:context" prompts plus `rows` requests whose contexts
are uniform in [lo, hi] and whose numbers of new tokens are uniform in [new_lo,
new_hi], all drawn from the case alone.
"""
import math
import random

import numpy as np
import torch

own = False

K_SCALE, V_SCALE = 0.02, 0.017


def _case(name, op, **kw):
    base = dict(op=op, prompts="", rows=0, lo=1, hi=1, new_lo=1, new_hi=1, len_seed=1, block=16)
    if op == "step":
        base.update(trees=True)
    else:
        base.update(heads=32, kv_heads=8, dim=128, e4m3=False)
        base.update(dict(padded=0.0) if op == "attend" else dict(layers=1, longest=4))
    base.update(kw)
    if name:
        base["name"] = name
    return base


def listed():
    return [
        # Four requests with a chain or tree of five tokens each: the latency of a small step's plan.
        _case("step few requests", "step", rows=4, lo=12, hi=700, new_lo=5, new_hi=5),
        # A large batch of drafted trees; some cross into new blocks.
        _case("step batch of trees", "step", rows=256, lo=16, hi=8192, new_lo=8, new_hi=24, len_seed=2),
        # Long prompts as they arrive together, and decoding requests; blocks of 32 tokens, no trees.
        _case("step long prompts", "step", prompts="8191:0,4097:1000,777:33,11000:0", rows=63, lo=256, hi=8192,
              len_seed=3, block=32, trees=False),
        # The smallest batch: short requests of a small model.
        _case("attend short", "attend", rows=4, lo=12, hi=37, new_lo=5, new_hi=5, heads=4, kv_heads=2, dim=64),
        # An 8B-shaped batch, small trees.
        _case("attend batch", "attend", rows=64, lo=512, hi=4096, new_lo=16, new_hi=16, len_seed=2),
        # The same with trees of 64 tokens: 256 query rows for each kv head.
        _case("attend large trees", "attend", rows=32, lo=512, hi=4096, new_lo=64, new_hi=64, len_seed=3),
        # Long contexts, few requests: the keys are split over the whole device.
        _case("attend long context", "attend", rows=8, lo=32000, hi=32768, new_lo=24, new_hi=32, len_seed=4),
        # Eight q heads per kv head over an e4m3 cache, ragged trees.
        _case("attend 70B e4m3", "attend", rows=96, lo=16, hi=4099, new_lo=1, new_hi=16, len_seed=5, heads=64,
              e4m3=True),
        # Odd head groups, blocks of 32, trees from one token to 130, a part of the rows padding.
        _case("attend ragged padded", "attend", rows=40, lo=0, hi=3000, new_lo=1, new_hi=130, len_seed=6, heads=28,
              kv_heads=4, block=32, padded=0.2),
        # One layer, few requests: the latency of a small commit.
        _case("commit one layer", "commit", rows=4, lo=12, hi=90, new_lo=8, new_hi=8),
        # All layers of an 8B-shaped model in one call.  (Short contexts keep the caches small: a commit
        # reads and writes the accepted rows alone.)
        _case("commit 32 layers", "commit", rows=64, lo=16, hi=120, new_lo=16, new_hi=32, len_seed=2, layers=32,
              longest=6),
        # e4m3 caches, many requests, odd lengths.
        _case("commit e4m3", "commit", rows=201, lo=1, hi=70, new_lo=9, new_hi=21, len_seed=3, layers=16, longest=7,
              block=32, e4m3=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "attend", "attend", "commit"])
    c = _case("", op, len_seed=rng.randrange(1 << 20), block=rng.choice([16, 16, 32, 64]))
    if op == "step":
        c["trees"] = rng.random() < 0.6
        c["rows"] = _log_uniform(rng, 1, 256)
        c["hi"] = _log_uniform(rng, 16, 8192)
        c["lo"] = rng.randint(1, c["hi"])
        c["new_hi"] = _log_uniform(rng, 1, 64)
        c["new_lo"] = rng.randint(0, c["new_hi"])
        if not c["trees"]:
            budget = 24000 - c["rows"] * c["new_hi"]
            prompts = []
            for _ in range(rng.randint(0, 4)):
                if budget < 100:
                    break
                n = _log_uniform(rng, 2, budget / 2)
                budget -= n
                prompts.append("%d:%d" % (n, rng.choice([0, rng.randint(1, 4000)])))
            c["prompts"] = ",".join(prompts)
        return c
    heads, kv_heads = rng.choice([(32, 8), (64, 8), (4, 2), (8, 8), (28, 4), (32, 2), (16, 1), (40, 8)])
    c.update(heads=heads, kv_heads=kv_heads, dim=rng.choice([64, 128, 128]), e4m3=rng.random() < 0.4)
    c["rows"] = _log_uniform(rng, 1, 128)
    if op == "commit":
        c["longest"] = rng.randint(1, 8)
        c["new_hi"] = rng.randint(c["longest"] + 1, 64)
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["hi"] = _log_uniform(rng, 2, 120)
        c["lo"] = rng.randint(1, c["hi"])
        values = c["rows"] * (c["hi"] + c["new_hi"] + c["block"]) * kv_heads * c["dim"]
        c["layers"] = max(1, _log_uniform(rng, 1, max(1, min(32, 200000000 // values))))
        return c
    c["new_hi"] = _log_uniform(rng, 1, 200)
    c["new_lo"] = rng.randint(1, c["new_hi"])
    c["padded"] = rng.choice([0.0, 0.0, 0.1])
    # no more keys and products than the long contexts' case
    most = min(260000 * 1024 // (kv_heads * c["dim"]), 260000 * 32 * 4096 // (c["new_hi"] * heads * c["dim"])) // c["rows"]
    c["hi"] = _log_uniform(rng, 1, max(16, min(32768, most)))
    c["lo"] = rng.randint(0, c["hi"])
    return c


def _batch(case):
    """Lengths, tree and accepted tokens of the case's requests (numpy): context_lens,
    new_lens, first row of each request; per row its parent in the request's tree (-1:
    the context), and the words of its ancestors' bits; accepted tokens."""
    rng = np.random.default_rng(case["len_seed"])
    prompts = [tuple(int(x) for x in t.split(":")) for t in case["prompts"].split(",") if t]
    ctx = np.concatenate([[c for _, c in prompts], rng.integers(case["lo"], case["hi"], case["rows"], endpoint=True)])
    new = np.concatenate([[n for n, _ in prompts],
                          rng.integers(case["new_lo"], case["new_hi"], case["rows"], endpoint=True)])
    ctx, new = ctx.astype(np.int64), new.astype(np.int64)
    first = np.concatenate([[0], np.cumsum(new)])
    b = dict(ctx=ctx, new=new, first=first, T=int(first[-1]))
    words = -(-case["new_hi"] // 64)
    if case["op"] == "commit":
        # Accepted tokens of each request, ascending.  Each stays where it is or comes from
        # behind the last accepted token's new place, so that a repeated pass finds the same values.
        b["accepted"] = np.zeros((len(ctx), case["longest"]), np.int64)
        b["counts"] = np.zeros(len(ctx), np.int64)
        for r in range(len(ctx)):
            n = int(rng.integers(0, case["longest"], endpoint=True))
            kept = int(rng.integers(0, n, endpoint=True))
            n = min(n, kept + max(0, int(new[r]) - n)) if n < new[r] else kept
            kept = min(kept, n, int(new[r]))
            n = min(n, int(new[r]))
            moved = n + np.sort(rng.permutation(int(new[r]) - n)[: n - kept])
            b["accepted"][r, :n] = np.concatenate([np.arange(n - len(moved)), moved])
            b["counts"][r] = n
        return b
    if case["op"] == "step" and not case["trees"]:
        return b
    parents = np.full(b["T"], -1, np.int64)
    bits = np.zeros((b["T"], words), np.uint64)
    depth = np.zeros(b["T"], np.int64)
    for r in range(len(ctx)):
        f, n = int(first[r]), int(new[r])
        for i in range(n):
            p = int(rng.integers(max(-1, i - 9), i)) if i else -1
            parents[f + i] = p
            if p >= 0:
                bits[f + i] = bits[f + p]
                depth[f + i] = depth[f + p] + 1
            bits[f + i, i // 64] |= np.uint64(1 << (i % 64))
        if case.get("padded"):  # the last rows of a tree of fixed size: they see nothing, nobody sees them
            live = n - int(n * case["padded"] * rng.random() * 2)
            bits[f + live:f + n] = 0
    b.update(parents=parents, bits=bits, depth=depth, words=words)
    return b


def _mask_tensor(bits):
    return torch.from_numpy(bits.view(np.int64).copy()).cuda()


def prepare(case, seed):
    b = _batch(case)
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B = case["block"]
    S = len(b["ctx"])

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(device=dev, dtype=torch.int32)

    total = -(-(b["ctx"] + b["new"]) // B)
    held = -(-b["ctx"] // B) if case["op"] == "step" else total
    mb = int(total.max()) + 1
    nb = int(total.sum()) + 1 + int(total.sum()) // 8
    perm = (torch.randperm(nb - 1, generator=gen, device=dev) + 1).to(torch.int32)  # block 0: the null block
    tables = torch.zeros(S, mb, dtype=torch.int32, device=dev)
    entered = torch.arange(mb, device=dev)[None, :] < torch.from_numpy(held).to(dev)[:, None]
    tables[entered] = perm[: int(held.sum())]
    s = dict(case=case, batch=b, tables=tables, context_lens=i32(b["ctx"]), query_lens=i32(b["new"]), nb=nb)
    if case["op"] == "step":
        free = torch.zeros(nb, dtype=torch.int32, device=dev)
        left = perm[int(held.sum()):]
        free[: len(left)] = left
        # buffers of a program that plans every step into the same ones, a few rows longer than this step
        T = b["T"] + 3
        s.update(held=i32(held), free=free, count=torch.tensor([len(left)], dtype=torch.int32, device=dev),
                 qsl=torch.zeros(S + 1, dtype=torch.int32, device=dev),
                 seq_lens=torch.zeros(S, dtype=torch.int32, device=dev),
                 slots=torch.zeros(T, dtype=torch.int64, device=dev),
                 positions=torch.zeros(T, dtype=torch.int32, device=dev), parents=None, masks=None)
        if case["trees"]:
            s["parents"] = i32(np.concatenate([b["parents"], np.full(3, -1)]))
            s["masks"] = torch.zeros(T, b["words"], dtype=torch.int64, device=dev)
        return s
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]

    def randn(*shape, mul=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * mul).to(torch.bfloat16)

    def cache(scale, *layers):
        x = randn(*layers, nb, B, hkv, d)
        return (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if case["e4m3"] else x

    if case["op"] == "commit":
        s.update(kc=cache(K_SCALE, case["layers"]), vc=cache(V_SCALE, case["layers"]), accepted=i32(b["accepted"]),
                 counts=i32(b["counts"]), new_lens=torch.zeros(S, dtype=torch.int32, device=dev))
        return s
    s.update(kc=cache(K_SCALE), vc=cache(V_SCALE), qsl=i32(b["first"]), seq_lens=i32(b["ctx"] + b["new"]),
             masks=_mask_tensor(b["bits"]), q=randn(b["T"], hq, d, mul=3.0),  # scores well beyond N(0, 1)
             scale=1.0 / math.sqrt(d), max_new=int(b["new"].max()), max_seq=int((b["ctx"] + b["new"]).max()))
    s["out"] = torch.empty_like(s["q"])
    s["ws"] = None
    if own:
        import paged_kv_cache_74_gb300 as pa
        s["ws"] = pa.new_workspace(pa.tree_workspace_size(S, b["T"], hq, hkv, d, s["max_seq"]), dev)
    return s


# ------------------------------------------------------------ the plain forms

def _plain_step(s):
    case, B = s["case"], s["case"]["block"]
    ctx, new, held, tables = s["context_lens"].long(), s["query_lens"].long(), s["held"].long(), s["tables"]
    S, T = len(ctx), len(s["slots"])
    dev = ctx.device
    first = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), new.cumsum(0)])
    seq = ctx + new
    # blocks: the i-th new one of the whole step is the i-th from the top of the stack
    need = ((seq + B - 1) // B - held).clamp(min=0)
    before = need.cumsum(0) - need
    j = torch.arange(tables.shape[1], device=dev) - held[:, None]
    fresh = (j >= 0) & (j < need[:, None])
    at = s["count"].long() - 1 - (before[:, None] + j)
    tables.copy_(torch.where(fresh, s["free"][at.clamp(0, len(s["free"]) - 1)], tables))
    taken = need.sum()
    # rows
    t = torch.arange(T, device=dev)
    r = (t[:, None] >= first[None, 1:]).sum(1)
    live = r < S
    r = r.clamp(max=S - 1)
    i = t - first[r]
    pos = torch.where(live, ctx[r] + i, 0)
    slots = tables[r, (pos // B).clamp(max=tables.shape[1] - 1)].long() * B + pos % B
    s["slots"].copy_(torch.where(live, slots, -1))
    if s["parents"] is not None:
        up = torch.where(live, s["parents"].long(), -1)
        masks = torch.zeros_like(s["masks"])
        depth = torch.full_like(t, -1)
        node = torch.where(live, i, -1)
        for _ in range(case["new_hi"]):  # one ancestor of every row at a time
            w = torch.arange(masks.shape[1], device=dev)
            bit = torch.bitwise_left_shift(torch.ones_like(node), node.clamp(min=0) % 64)
            masks |= torch.where((node[:, None] // 64 == w) & (node[:, None] >= 0), bit[:, None], 0)
            depth += node >= 0
            node = torch.where(node >= 0, up[(first[r] + node).clamp(0, T - 1)], -1)
        s["masks"].copy_(masks)
        pos = torch.where(live, ctx[r] + depth, 0)
    s["positions"].copy_(pos)
    s["qsl"].copy_(first)
    s["seq_lens"].copy_(seq)
    held = held + need
    # what the step did not keep goes back, so that the last block taken lies deepest
    left = s["count"].long() - taken
    keep = (ctx + B - 1) // B
    back = (held - keep).clamp(min=0)
    gone = back.sum()
    j = torch.arange(tables.shape[1], device=dev) - keep[:, None]
    freed = (j >= 0) & (j < back[:, None])
    at = left + gone - 1 - ((back.cumsum(0) - back)[:, None] + j)
    s["free"].index_put_((torch.where(freed, at, len(s["free"]) - 1).flatten(),),
                         torch.where(freed, tables, s["free"][-1]).flatten())
    s["count"].copy_(left + gone)
    s["held"].copy_(held - back)


def _values(codes, scale):
    """A cache's values in 32 bits."""
    return codes.view(torch.float8_e4m3fn).float() * scale if codes.dtype == torch.uint8 else codes.float()


def _plain_attend(s):
    case, b, B = s["case"], s["batch"], s["case"]["block"]
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    for r in range(len(b["ctx"])):
        f, n, ctx = int(b["first"][r]), int(b["new"][r]), int(b["ctx"][r])
        ids = s["tables"][r, : -(-(ctx + n) // B)].long()
        k = _values(s["kc"][ids], K_SCALE).flatten(0, 1)[: ctx + n].permute(1, 2, 0)
        v = _values(s["vc"][ids], V_SCALE).flatten(0, 1)[: ctx + n].transpose(0, 1)
        q = s["q"][f:f + n].float().view(n, hkv, hq // hkv, d).transpose(0, 1).reshape(hkv, -1, d)
        x = (q @ k).view(hkv, n, hq // hkv, ctx + n) * s["scale"]
        node = torch.arange(n, device=q.device)
        seen = (s["masks"][f:f + n][:, node // 64] >> (node % 64)) & 1
        # (a row whose mask is empty still sees the context, if there is one)
        x[..., ctx:] = x[..., ctx:].masked_fill(seen[:, None] == 0, -math.inf)
        m = x.amax(-1, keepdim=True)
        w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
        o = (w.reshape(hkv, -1, ctx + n) @ v).view(hkv, n, -1, d).transpose(0, 1)
        s["out"][f:f + n] = o.reshape(n, hq, d).to(torch.bfloat16)
    return s["out"]


def _plain_commit(s):
    B = s["case"]["block"]
    ctx, counts = s["context_lens"].long(), s["counts"].long()
    i = torch.arange(s["accepted"].shape[1], device=ctx.device)
    r, at = torch.nonzero(i < counts[:, None], as_tuple=True)
    place = []
    for pos in (ctx[r] + s["accepted"][r, at], ctx[r] + at):
        place.append(s["tables"][r, pos // B].long() * B + pos % B)
    for c in (s["kc"], s["vc"]):
        rows = c.flatten(1, 2)
        rows[:, place[1]] = rows[:, place[0]]
    s["new_lens"].copy_(ctx + counts)


def run(s):
    case = s["case"]
    if own:
        import paged_kv_cache_74_gb300 as pa
    if case["op"] == "step":
        if own:
            pa.plan_step(s["tables"], s["held"], s["context_lens"], s["query_lens"], s["free"], s["count"],
                         case["block"], s["nb"], s["qsl"], s["seq_lens"], s["slots"], s["positions"],
                         parents=s["parents"], tree_masks=s["masks"])
            pa.release_blocks(s["tables"], s["held"], s["context_lens"], s["free"], s["count"], case["block"], s["nb"])
        else:
            _plain_step(s)
        names = ["tables", "held", "free", "count", "qsl", "seq_lens", "slots", "positions"]
        return {n: s[n] for n in names + (["masks"] if case["trees"] else [])}
    if case["op"] == "commit":
        if own:
            pa.commit_tokens(s["kc"], s["vc"], s["tables"], s["context_lens"], s["query_lens"], s["accepted"],
                             s["counts"], new_lens=s["new_lens"])
        else:
            _plain_commit(s)
        kept = (s["kc"], s["vc"])
        if case["e4m3"]:
            kept = tuple(c.view(torch.float8_e4m3fn) for c in kept)
        return {"key_cache": kept[0], "value_cache": kept[1], "new_lens": s["new_lens"]}
    if not own:
        return _plain_attend(s)
    call, scales = (pa.tree_attention_fp8, (K_SCALE, V_SCALE)) if case["e4m3"] else (pa.tree_attention, ())
    return call(s["q"], s["kc"], s["vc"], s["qsl"], s["seq_lens"], s["tables"], s["masks"], s["max_new"],
                s["max_seq"], s["scale"], *scales, out=s["out"], workspace=s["ws"])


def work(case):
    b = _batch(case)
    B, S, T = case["block"], len(b["ctx"]), b["T"]
    if case["op"] == "step":
        blocks = int((-(-(b["ctx"] + b["new"]) // B) + -(-b["ctx"] // B) * -1).sum())
        # lengths, held counts and offsets; each new block: read and entered, and back; the rows' slots,
        # positions and, with trees, parents and masks; the block ids of the new rows
        rows = T * (8 + 4 + ((4 + 8 * b["words"]) if case["trees"] else 0))
        return {"bytes": 4 * (7 * S + 1) + 16 * blocks + rows, "flops": 0}
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    element = 1 if case["e4m3"] else 2
    if case["op"] == "commit":
        moved = int((b["accepted"] != np.arange(case["longest"]))[np.arange(case["longest"]) < b["counts"][:, None]].sum())
        return {"bytes": case["layers"] * moved * hkv * d * element * 2 * 2 + 4 * int(b["counts"].sum()) + 12 * S,
                "flops": 0}
    keys = int((b["ctx"] + b["new"]).sum())
    seen = int(sum(bin(int(w)).count("1") for w in b["bits"].flatten()))
    pairs = float((b["ctx"] * b["new"]).sum()) + seen
    return {"bytes": keys * hkv * d * 2 * element + T * hq * d * 4 + T * 8 * b["words"] + 4 * (keys // B) + 8 * S,
            "flops": 4.0 * d * hq * pairs}


# ------------------------------------------------ the definitions, in 64 bits

def _exact_step(s):
    """The step in Python integers: a list of free blocks, popped and pushed one at a time."""
    case, b, B = s["case"], s["batch"], s["case"]["block"]
    tables = s["tables"].cpu().numpy().astype(np.int64)
    held = [int(x) for x in s["held"].cpu()]
    room = s["free"].cpu().numpy().astype(np.int64)
    stack = list(room[: int(s["count"])])
    T = len(s["slots"])
    slots, positions = np.full(T, -1, np.int64), np.zeros(T, np.int64)
    masks = np.zeros((T, b["words"]), np.uint64) if case["trees"] else None
    for r, (ctx, new) in enumerate(zip(b["ctx"], b["new"])):
        while held[r] * B < ctx + new:
            tables[r, held[r]] = stack.pop()
            held[r] += 1
        for i in range(new):
            t = b["first"][r] + i
            slots[t] = tables[r, (ctx + i) // B] * B + (ctx + i) % B
            positions[t] = ctx + (b["depth"][t] if case["trees"] else i)
            if case["trees"]:
                masks[t] = b["bits"][t]
    for r in reversed(range(len(held))):  # the last block taken goes back first
        while held[r] > -(-int(b["ctx"][r]) // B):
            held[r] -= 1
            stack.append(tables[r, held[r]])
    room[: len(stack)] = stack
    out = dict(tables=tables, held=np.array(held), free=room, count=np.array([len(stack)]), qsl=b["first"],
               seq_lens=b["ctx"] + b["new"], slots=slots, positions=positions)
    if case["trees"]:
        out["masks"] = masks.view(np.int64)
    return {n: torch.from_numpy(np.ascontiguousarray(x)).cuda() for n, x in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    b, B = s["batch"], case["block"]
    if case["op"] == "step":
        return _exact_step(s)
    if case["op"] == "commit":
        tables = s["tables"].cpu().numpy()
        for r in range(len(b["ctx"])):
            for i in range(int(b["counts"][r])):
                src, dst = int(b["ctx"][r] + b["accepted"][r, i]), int(b["ctx"][r] + i)
                for c in (s["kc"], s["vc"]):
                    c[:, int(tables[r, dst // B]), dst % B] = c[:, int(tables[r, src // B]), src % B].clone()
        kept = [(c.view(torch.float8_e4m3fn) if case["e4m3"] else c).double() for c in (s["kc"], s["vc"])]
        return {"key_cache": kept[0], "value_cache": kept[1],
                "new_lens": torch.from_numpy(b["ctx"] + b["counts"]).cuda()}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    tables = s["tables"].cpu().numpy().astype(np.int64)
    for r in range(len(b["ctx"])):
        f, n, ctx = int(b["first"][r]), int(b["new"][r]), int(b["ctx"][r])
        where = np.arange(ctx + n)
        where = torch.from_numpy(tables[r, where // B] * B + where % B).cuda()
        seen = np.ones((n, ctx + n), bool)
        for i in range(n):
            for j in range(n):
                seen[i, ctx + j] = bool(int(b["bits"][f + i, j // 64]) >> (j % 64) & 1)
        seen = torch.from_numpy(seen).cuda()[:, None]
        kv = []
        for codes, scale in ((s["kc"], K_SCALE), (s["vc"], V_SCALE)):
            x = codes.flatten(0, 1)[where]
            kv.append(x.view(torch.float8_e4m3fn).double() * scale if case["e4m3"] else x.double())
        for h in range(case["kv_heads"]):
            hs = slice(h * group, (h + 1) * group)
            e = torch.einsum("rgd,jd->rgj", s["q"][f:f + n, hs].double(), kv[0][:, h]) / math.sqrt(case["dim"])
            e = torch.where(seen, e, -math.inf)
            weight = torch.where(seen, torch.exp(e - torch.logsumexp(e, -1, keepdim=True)), 0.0)
            out[f:f + n, hs] = torch.einsum("rgj,jd->rgd", weight, kv[1][:, h])
    return out
