"""Measured cases of the calls for paged caches that many requests share or that outgrow the memory:
decoding of requests that share a prefix, the attention weight that cached tokens gather, the choice
of the tokens that stay, and the move of those to the front of their pages.

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it makes
the library's calls."""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------ cases
def _shared(name, reqs, groups, prefix, suffix, hq, hkv, q_len=1, fmt="token", block=16, gates=False, window=0,
            sink=False, nhd=False):
    """`groups` of about reqs / groups requests that share up to `prefix` tokens each, with up to
    `suffix` tokens of their own behind them (the query rows among those)."""
    return dict(name=name, op="shared", reqs=reqs, groups=groups, prefix=prefix, suffix=suffix, hq=hq, hkv=hkv, d=128,
                q_len=q_len, fmt=fmt, block=block, gates=gates, window=window, sink=sink, nhd=nhd)


def _weights(name, reqs, q_len, ctx, hq, hkv, d, fmt="token", block=16, gates=False, window=0, sink=False, nhd=False,
             decay=1.0, lse=False):
    """The last q_len rows of contexts up to `ctx`; lse: the rows' sums of exponentials are at hand."""
    return dict(name=name, op="weights", reqs=reqs, q_len=q_len, ctx=ctx, hq=hq, hkv=hkv, d=d, fmt=fmt, block=block,
                gates=gates, window=window, sink=sink, nhd=nhd, decay=decay, lse=lse)


def _select(name, reqs, ctx, hkv, keep, block=16, first=0, recent=0):
    return dict(name=name, op="select", reqs=reqs, ctx=ctx, hkv=hkv, keep=keep, block=block, first=first,
                recent=recent)


def _compact(name, reqs, ctx, hq, hkv, d, keep, fmt="token", block=16, gates=False, nhd=False):
    return dict(name=name, op="compact", reqs=reqs, ctx=ctx, hq=hq, hkv=hkv, d=d, keep=keep, fmt=fmt, block=block,
                gates=gates, nhd=nhd)


def listed():
    return [
        # a few requests behind one short system prompt: latency
        _shared("shared_4x1_2048", 4, 1, 2048, 64, 16, 1),
        # a serving batch behind one long prompt, each with a conversation of its own
        _shared("shared_64x1_16384", 64, 1, 16384, 2048, 64, 4),
        # three prompts of an odd length, drafts of four tokens to verify, bf16 cache with gates and sinks
        _shared("shared_bf16_48x4_30011", 48, 3, 30011, 512, 32, 4, q_len=4, fmt="bf16", block=64, gates=True,
                sink=True, nhd=True),
        # each decoding step's weights added to what the cached tokens have gathered
        _weights("weights_decode_64x1", 64, 1, 32768, 64, 4, 128),
        # the last rows of prompts look back over them: wide heads, bf16, gates
        _weights("weights_last_8x33_d256", 8, 33, 16384, 16, 4, 256, fmt="bf16", block=32, gates=True, decay=0.0),
        # chunks of a prefill: every row counts
        _weights("weights_chunk_4x1024", 4, 1024, 32768, 64, 4, 128),
        # a few short contexts
        _select("select_3x300", 3, 300, 1, 64, first=4, recent=16),
        # a serving batch goes back to 4096 tokens a request
        _select("select_64x32768", 64, 32768, 4, 4096, first=4, recent=64),
        # two very long contexts
        _select("select_2x227000", 2, 227000, 4, 16384, block=64, first=16, recent=256),
        # a few short contexts of small heads
        _compact("compact_3x300_d64", 3, 300, 8, 1, 64, 64),
        # the serving batch's pages, with gates
        _compact("compact_64x32768", 64, 32768, 64, 4, 128, 4096, gates=True),
        # wide heads in bf16, slots outside the heads
        _compact("compact_bf16_8x16384_d256", 8, 16384, 16, 4, 256, 4096, fmt="bf16", block=32, nhd=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = [work(c) for c in listed()]
    most = {k: max(w[k] for w in top) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["shared", "shared", "weights", "weights", "select", "compact"])
        fmt = rng.choice(["token", "token", "tensor", "bf16"])
        hkv, block = rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 64, 128])
        reqs, nhd = _log_int(rng, 1, 64), rng.random() < 0.5
        gates, sink = rng.random() < 0.4, rng.random() < 0.3
        window = _log_int(rng, 16, 16384) if rng.random() < 0.25 else 0
        if op == "shared":
            c = _shared("", reqs, min(reqs, _log_int(rng, 1, 6)), _log_int(rng, 1, 32768), _log_int(rng, 4, 4096),
                        hkv * rng.choice([8, 16]), hkv, rng.choice([1, 1, 1, 2, 3, 4]), fmt, block, gates, window,
                        sink, nhd)
        elif op == "weights":
            d, ctx = rng.choice([64, 128, 128, 256, 512]), _log_int(rng, 1, 32768)
            c = _weights("", reqs, min(ctx, _log_int(rng, 1, 1024)), ctx, hkv * rng.choice([1, 2, 4, 7, 8, 16]), hkv,
                         d, fmt, block, gates, window, sink, nhd, rng.choice([0.0, 0.9, 1.0]), rng.random() < 0.2)
        elif op == "select":
            ctx = _log_int(rng, 32, 227000)
            keep = _log_int(rng, 8, min(ctx - 8, 16384))
            c = _select("", reqs, ctx, hkv, keep, block, min(rng.choice([0, 4, 16]), keep // 4),
                        min(rng.choice([0, 16, 256]), keep // 4))
        else:
            ctx = _log_int(rng, 1, 32768)
            c = _compact("", reqs, ctx, hkv * rng.choice([1, 2, 4, 7, 8]), hkv, rng.choice([64, 128, 128, 256, 512]),
                         _log_int(rng, 1, ctx), fmt, block, gates, nhd)
        del c["name"]
        w = work(c)
        # the cache stays within a few GB
        if op in ("weights", "compact") and reqs * c["ctx"] * (hkv * c["d"] * 2 + c["hq"]) > 1 << 31:
            continue
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


# ----------------------------------------------------------------------------------------- inputs
def _share(i, n, top):
    """A length up to `top` for the i-th of n, from the case alone: the last has it whole."""
    return top if i == n - 1 else max(1, int(top * ((i * 5 + 4) % 13 + 1) / 13.0))


def _lengths(case):
    """(cached tokens, query rows) of each request."""
    n = case["reqs"]
    if case["op"] == "shared":
        lens, rows = [], []
        first, prefix = _groups(case)
        for g, p in enumerate(prefix):
            for i in range(first[g], first[g + 1]):
                ql = 1 + (case["q_len"] - 1 - i) % case["q_len"]
                rows.append(ql)
                lens.append(p + max(ql, _share(i, n, case["suffix"])))
        return lens, rows
    lens = [_share(i, n, case["ctx"]) for i in range(n)]
    return lens, [min(x, case.get("q_len", 0)) for x in lens]


def _groups(case):
    """(first request of each group and the end, shared tokens of each group)."""
    n, g = case["reqs"], case["groups"]
    return [n * i // g for i in range(g + 1)], [_share(i, g, case["prefix"]) for i in range(g)]


def _kept(case):
    """Tokens that stay of each request."""
    return [min(x, _share(i, case["reqs"], case["keep"])) for i, x in enumerate(_lengths(case)[0])]


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _heads(gen, tokens, heads, d, dev):
    """A projection's output: tokens and heads of different sizes, some dims larger than others."""
    x = torch.randn((tokens, heads, d), generator=gen, device=dev)
    x *= torch.exp(0.3 * torch.randn((tokens, heads, 1), generator=gen, device=dev))
    x *= torch.exp(0.3 * torch.randn((1, heads, d), generator=gen, device=dev))
    return x


def _pages(gen, case, lens, dev):
    """(block table, blocks of the cache); with shared prefixes their whole blocks belong to the group."""
    block, n = case["block"], len(lens)
    need = [-(-x // block) for x in lens]
    common = [0] * n
    if case["op"] == "shared":
        first, prefix = _groups(case)
        for g, p in enumerate(prefix):
            for i in range(first[g] + 1, first[g + 1]):
                common[i] = p // block
    nb = sum(need) - sum(common) + 8
    perm = torch.randperm(nb, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((n, max(need)), dtype=torch.int32, device=dev)
    at = 0
    for i in range(n):
        if common[i]:
            table[i, :common[i]] = table[i - 1, :common[i]]
        table[i, common[i]:need[i]] = perm[at:at + need[i] - common[i]]
        at += need[i] - common[i]
    return table, nb


def _cache(gen, case, nb, dev):
    shape = (nb, case["block"], case["hkv"], case["d"])
    if not case["nhd"]:
        shape = (nb, case["hkv"], case["block"], case["d"])
    x = torch.empty(shape, dtype=torch.bfloat16 if case["fmt"] == "bf16" else torch.uint8, device=dev)
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, nb, step):
        y = torch.randn((min(step, nb - i),) + shape[1:], generator=gen, device=dev)
        if case["fmt"] == "bf16":
            x[i:i + step] = y.to(torch.bfloat16)
        else:
            x[i:i + step] = (y * 100.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.permute(0, 2, 1, 3) if case["nhd"] else x


def _scale(gen, case, nb, dev):
    if case["fmt"] == "token":  # a spread of four
        return torch.exp(torch.rand((nb, case["hkv"], case["block"]), generator=gen, device=dev) * math.log(4.0)) / 200
    if case["fmt"] == "tensor":  # one for the whole cache, from a calibration
        return torch.rand((1,), generator=gen, device=dev) * 0.005 + 0.008
    return None


def _gates(gen, case, table, nb, lens, dev):
    """Cumulative log gates of each request: about -0.004 a token."""
    g = torch.zeros((nb, case["hq"], case["block"]), device=dev)
    top, runs = max(lens), []
    z = 6.0 + torch.randn((top, case["hq"]), generator=gen, device=dev)
    c = (-torch.log1p(torch.exp(-z))).cumsum(0, dtype=torch.float64).float()
    pad = -(-top // case["block"]) * case["block"] - top
    pages = torch.nn.functional.pad(c, (0, 0, 0, pad)).view(-1, case["block"], case["hq"]).transpose(1, 2)
    for i, x in enumerate(lens):  # one run of gates: shared blocks get the same from each of their requests
        n = -(-x // case["block"])
        g[table[i, :n].long()] = pages[:n]
    return g


def _gathered(gen, nb, hkv, block, dev):
    """Weights that tokens have gathered so far: a few large ones, and some that nothing ever looked at."""
    w = torch.exp(2.0 * torch.randn((nb, hkv, block), generator=gen, device=dev) - 4.0)
    return w * (torch.rand((nb, hkv, block), generator=gen, device=dev) > 0.05)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case)
    lens, rows = _lengths(case)
    hkv, block = case["hkv"], case["block"]
    s["lens"], s["max_seq_len"] = lens, max(lens)
    s["table"], nb = _pages(gen, case, lens, dev)
    s["seq_lens"] = _i32(lens, dev)
    if case["op"] != "shared":
        s["w"] = _gathered(gen, nb, hkv, block, dev)
    if case["op"] in ("select", "compact"):
        s["keep_each"] = _kept(case)
    if case["op"] == "select":
        s["budgets"] = _i32(s["keep_each"], dev)
        s["first_lens"] = _i32([case["first"]] * case["reqs"], dev) if case["first"] else None
        return s
    s["k_cache"], s["k_scale"] = _cache(gen, case, nb, dev), _scale(gen, case, nb, dev)
    s["g_cache"] = _gates(gen, case, s["table"], nb, lens, dev) if case["gates"] else None
    if case["op"] != "weights":
        s["v_cache"], s["v_scale"] = _cache(gen, case, nb, dev), _scale(gen, case, nb, dev)
    if case["op"] == "compact":
        keep = s["keep_each"]
        s["kept"] = torch.full((case["reqs"], hkv, max(keep)), -1, dtype=torch.int32, device=dev)
        for i, (x, n) in enumerate(zip(lens, keep)):  # a random choice for every head
            u = torch.rand((hkv, x), generator=gen, device=dev)
            s["kept"][i, :, :n] = u.topk(n, 1).indices.sort(1).values.to(torch.int32)
        s["kept_lens"] = _i32(keep, dev)
        return s
    cu = [0]
    for x in rows:
        cu.append(cu[-1] + x)
    s["cu"], s["rows"], s["first_row"], s["max_q_len"] = _i32(cu, dev), rows, cu, max(rows)
    s["q"] = _heads(gen, cu[-1], case["hq"], case["d"], dev).to(torch.bfloat16)
    s["sinks"] = torch.randn(case["hq"], generator=gen, device=dev) if case["sink"] else None
    s["scale"] = case["d"] ** -0.5
    if case["op"] == "shared":
        first, prefix = _groups(case)
        s["first"], s["shared_len"] = first, prefix
        s["cu_groups"], s["prefix_lens"] = _i32(first, dev), _i32(prefix, dev)
        for g, p in enumerate(prefix):  # the tokens of a block that the prefix fills in part are in each request's own
            b = p % case["block"]
            last = s["table"][first[g]:first[g + 1], p // case["block"] if b else 0].long()
            for t in (s["k_cache"], s["v_cache"]) + ((s["k_scale"], s["v_scale"]) if case["fmt"] == "token" else ()):
                t[last[1:], :, :b] = t[last[:1], :, :b]
        s["group_q"] = max(cu[first[g + 1]] - cu[first[g]] for g in range(len(prefix)))
        s["max_prefix"] = max(prefix)
        s["max_suffix"] = max(lens[i] - p for g, p in enumerate(prefix) for i in range(first[g], first[g + 1]))
    else:
        s["sums"] = None
        if case["lse"]:
            s["sums"] = torch.empty((case["hq"], cu[-1]), device=dev)
            for i in range(case["reqs"]):
                for h in range(hkv):
                    z = torch.logsumexp(_joined(s, i, h)[0], -1)
                    s["sums"].view(hkv, -1, cu[-1])[h, :, cu[i]:cu[i + 1]] = z.view(-1, rows[i]) if rows[i] else 0.0
    return s


# ------------------------------------------------------------------------------------- plain forms
def _blocks(s, i, a, b):
    """Blocks of the positions [a, b) of request i, and where in them they are."""
    p = torch.arange(a, b, device=s["table"].device)
    return s["table"][i][p // s["block"]].long(), p % s["block"]


def _read(cache, scale, fmt, blk, slot, h):
    x = cache[blk, h, slot]
    if fmt == "bf16":
        return x.float()
    x = x.view(torch.float8_e4m3fn).float()
    return x * (scale[blk, h, slot][:, None] if fmt == "token" else scale)


def _scores(s, i, h, q, pos, a, b):
    """Scores [G, rows, b - a] of rows at `pos` of head group h over the positions [a, b) of request i.
    q [rows, G, d]; the rows' own cumulative gates [rows, G] come with it."""
    blk, slot = _blocks(s, i, a, b)
    q, own_gate = q
    x = (q.float().transpose(0, 1) @ _read(s["k_cache"], s["k_scale"], s["fmt"], blk, slot, h).T) * s["scale"]
    if own_gate is not None:
        g = s["g_cache"].view(s["g_cache"].shape[0], s["hkv"], -1, s["block"])[blk, h, :, slot]  # [keys, G]
        x = x + (own_gate.T[:, :, None] - g.T[:, None, :])
    j = torch.arange(a, b, device=q.device)
    seen = j <= pos[:, None]
    if s["window"]:
        seen &= j > pos[:, None] - s["window"]
    return x.masked_fill_(~seen, -math.inf)


def _rows_of(s, i, h):
    """Query rows [rows, G, d] of request i and head group h with their own gates, and their positions."""
    a, n = s["first_row"][i], s["rows"][i]
    q = s["q"][a:a + n].unflatten(1, (s["hkv"], -1))[:, h]
    pos = torch.arange(s["lens"][i] - n, s["lens"][i], device=q.device)
    gate = None
    if s["g_cache"] is not None:
        blk, slot = _blocks(s, i, s["lens"][i] - n, s["lens"][i])
        gate = s["g_cache"].view(s["g_cache"].shape[0], s["hkv"], -1, s["block"])[blk, h, :, slot]
    return (q, gate), pos


def _joined(s, i, h):
    """Scores [G, rows, keys (and the sink)] of request i and head group h, and its keys."""
    q, pos = _rows_of(s, i, h)
    x, n = _scores(s, i, h, q, pos, 0, s["lens"][i]), s["lens"][i]
    if s["sinks"] is not None:
        x = torch.cat([x, s["sinks"].view(s["hkv"], -1)[h][:, None, None].expand(-1, x.shape[1], 1)], -1)
    return x, n


def _shared_plain(s):
    out = torch.empty_like(s["q"])
    o = out.unflatten(1, (s["hkv"], -1))
    for g, p in enumerate(s["shared_len"]):
        ids = range(s["first"][g], s["first"][g + 1])
        for h in range(s["hkv"]):
            each = [_rows_of(s, i, h) for i in ids]
            q = torch.cat([x[0][0] for x in each])
            gate = torch.cat([x[0][1] for x in each]) if s["g_cache"] is not None else None
            blk, slot = _blocks(s, ids[0], 0, p)
            v = _read(s["v_cache"], s["v_scale"], s["fmt"], blk, slot, h)
            x = _scores(s, ids[0], h, (q, gate), torch.cat([x[1] for x in each]), 0, p)  # [G, all rows, p]
            top = x.amax(-1).clamp_(min=-1e30)
            x = torch.exp(x - top[..., None])
            den, acc, at = x.sum(-1), x @ v, 0
            for i, (qi, pos) in zip(ids, each):
                n = s["rows"][i]
                blk, slot = _blocks(s, i, p, s["lens"][i])
                y = _scores(s, i, h, qi, pos, p, s["lens"][i])
                m = torch.maximum(top[:, at:at + n], y.amax(-1))
                if s["sinks"] is not None:
                    sink = s["sinks"].view(s["hkv"], -1)[h][:, None]
                    m = torch.maximum(m, sink)
                y, w = torch.exp(y - m[..., None]), torch.exp(top[:, at:at + n] - m)
                d = den[:, at:at + n] * w + y.sum(-1)
                if s["sinks"] is not None:
                    d = d + torch.exp(sink - m)
                z = acc[:, at:at + n] * w[..., None] + y @ _read(s["v_cache"], s["v_scale"], s["fmt"], blk, slot, h)
                o[s["first_row"][i]:s["first_row"][i] + n, h] = (z / d[..., None]).transpose(0, 1).to(torch.bfloat16)
                at += n
    return out


def _weights_plain(s):
    for i in range(s["reqs"]):
        n, new = s["lens"][i], s["rows"][i]
        blk, slot = _blocks(s, i, 0, n)
        for h in range(s["hkv"]):
            x, _ = _joined(s, i, h)
            if s["sums"] is None:
                x -= x.amax(-1, keepdim=True)
                x.exp_()
                x /= x.sum(-1, keepdim=True)
            else:
                a = s["first_row"][i]
                x -= s["sums"].view(s["hkv"], -1, s["sums"].shape[1])[h, :, a:a + new, None]
                x.exp_()
            w = x[..., :n].sum((0, 1))
            if s["decay"]:
                w[:n - new] += s["decay"] * s["w"][blk[:n - new], h, slot[:n - new]]
            s["w"][blk, h, slot] = w
    return s["w"]


def _chosen(s, weights):
    """kept and kept_lens, with the weights of request i and all its heads, [hkv, tokens]."""
    dev, keep = s["table"].device, s["keep_each"]
    kept = torch.full((s["reqs"], s["hkv"], s["keep"]), -1, dtype=torch.int32, device=dev)
    for i in range(s["reqs"]):
        x, n = s["lens"][i], min(keep[i], s["lens"][i])
        last = min(n, s["recent"])
        lead = min(n - last, s["first"], x - last)
        mid = weights(i)[:, lead:x - last]
        # ties go to the lowest index
        best = mid.sort(dim=1, descending=True, stable=True).indices[:, :n - last - lead].sort(1).values + lead
        kept[i, :, :lead] = torch.arange(lead, device=dev)
        kept[i, :, lead:n - last] = best
        kept[i, :, n - last:n] = torch.arange(x - last, x, device=dev)
    return kept, torch.minimum(s["budgets"], s["seq_lens"])


def _row_weights(s, i):
    blk, slot = _blocks(s, i, 0, s["lens"][i])
    return s["w"][blk, :, slot].T


def _moved(s):
    """The tensors that go along with the tokens: [blocks, heads, slots, ...], heads a multiple of hkv."""
    t = dict(k=s["k_cache"], v=s["v_cache"], w=s["w"])
    if s["fmt"] == "token":
        t.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["g_cache"] is not None:
        t["g"] = s["g_cache"]
    return t


def _compact_plain(s):
    keep = s["keep_each"]
    for t in _moved(s).values():
        t = t.unflatten(1, (s["hkv"], -1))  # [blocks, hkv, heads each, slots, ...]
        for i in range(s["reqs"]):
            to, slot = _blocks(s, i, 0, keep[i])
            src = s["kept"][i, :, :keep[i]].long()
            for h in range(s["hkv"]):
                t[to, h, :, slot] = t[s["table"][i][src[h] // s["block"]].long(), h, :, src[h] % s["block"]]


def run(s):
    if own:
        import gated_causal_softmax_gb300 as gcs
    if s["op"] == "shared":
        if not own:
            return _shared_plain(s)
        return gcs.attn_decode_paged_shared(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                            s["seq_lens"], s["cu"], s["max_q_len"], s["max_seq_len"], s["cu_groups"],
                                            s["prefix_lens"], s["group_q"], s["max_prefix"], s["max_suffix"],
                                            s["scale"], g_cache=s["g_cache"], sink=s["sinks"], window=s["window"])
    if s["op"] == "weights":
        if not own:
            return _weights_plain(s)
        return gcs.attn_cache_weights(s["q"], s["k_cache"], s["k_scale"], s["table"], s["seq_lens"], s["cu"],
                                      s["max_q_len"], s["max_seq_len"], s["w"], s["decay"], s["sums"], s["scale"],
                                      g_cache=s["g_cache"], sink=s["sinks"], window=s["window"])
    if s["op"] == "select":
        if not own:
            return _chosen(s, lambda i: _row_weights(s, i))
        return gcs.attn_cache_select(s["w"], s["table"], s["seq_lens"], s["max_seq_len"], s["budgets"], s["keep"],
                                     s["first_lens"], s["recent"])
    if own:
        gcs.attn_cache_compact(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["seq_lens"],
                               s["kept"], s["kept_lens"], g_cache=s["g_cache"], w_cache=s["w"])
    else:
        _compact_plain(s)
    return {k: t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for k, t in _moved(s).items()}


# ------------------------------------------------------------------------------------------- work
def _seen(case, n, rows):
    """(pairs of a row and a key that it sees, keys that any row sees) of one request and head."""
    w = case["window"] or n
    if n - rows + 1 >= w:
        return rows * w, min(n, rows + w - 1)
    return sum(min(w, p + 1) for p in range(n - rows, n)), n


def work(case):
    lens, rows = _lengths(case)
    n, hkv = case["reqs"], case["hkv"]
    pages = sum(-(-x // case["block"]) for x in lens)
    if case["op"] == "select":
        keep = _kept(case)
        return {"bytes": 4 * (hkv * sum(lens) + n * hkv * case["keep"] + pages + 3 * n), "flops": hkv * sum(lens)}
    hq, d = case["hq"], case["d"]
    held, extra = (2 if case["fmt"] == "bf16" else 1), (4 if case["fmt"] == "token" else 0)
    gate = 4 * hq if case["gates"] else 0
    if case["op"] == "compact":
        moved = 2 * hkv * (d * held + extra) + 4 * hkv + gate
        return {"bytes": sum(_kept(case)) * (2 * moved + 4 * hkv) + 4 * pages, "flops": 0}
    seen = [_seen(case, x, r) for x, r in zip(lens, rows)]
    pairs, keys = sum(x for x, _ in seen) * hq, sum(x for _, x in seen)
    q_bytes = 2 * sum(rows) * hq * d
    if case["op"] == "weights":
        b = keys * (hkv * (d * held + extra) + gate) + q_bytes + 4 * pages
        b += 4 * hkv * sum(lens) * (2 if case["decay"] else 1) + (4 * hq * sum(rows) if case["lse"] else 0)
        return {"bytes": b, "flops": 2 * d * pairs}
    first, prefix = _groups(case)
    for g, p in enumerate(prefix):  # shared keys count once a group
        read = [max(0, p - (lens[i] - seen[i][1])) for i in range(first[g], first[g + 1])]
        keys -= sum(read) - max(read)
    return {"bytes": keys * (2 * hkv * (d * held + extra) + gate) + 2 * q_bytes + 4 * pages, "flops": 4 * d * pairs}


# ------------------------------------------------------------------------------- values in 64 bits
def _wide(t, block, hkv):
    """[blocks, heads, slots, ...] -> a copy [hkv, heads each, blocks * slots, ...] in 64 bits."""
    if t.dtype == torch.uint8:
        t = t.view(torch.float8_e4m3fn)
    t = t.to(torch.float64).transpose(0, 1)
    return t.reshape((hkv, -1, t.shape[1] * block) + tuple(t.shape[3:]))


def _cells(s, i, dev):
    p = torch.arange(s["lens"][i], device=dev)
    return s["table"][i].long()[p // s["block"]] * s["block"] + p % s["block"]


def _weights_of(s, i, h, keys, gates, lse):
    """exp(score - lse) of every row over a request's keys in 64 bits, [rows, G, keys]: `keys` [n, d];
    with lse None the rows' own sums, the sink among them."""
    a, r, n = s["first_row"][i], s["rows"][i], s["lens"][i]
    dev, G = keys.device, s["hq"] // s["hkv"]
    q = s["q"][a:a + r, h * G:(h + 1) * G].double()
    x = torch.einsum("rgd,nd->rgn", q, keys) * s["scale"]
    if gates is not None:
        x += gates[:, n - r:].T[..., None] - gates[None]
    back = torch.arange(n - r, n, device=dev)[:, None] - torch.arange(n, device=dev)[None]
    hide = (back < 0) | (back >= s["window"]) if s["window"] else back < 0
    x.masked_fill_(hide[:, None], -math.inf)
    if lse is None:
        lse = torch.logsumexp(x, -1)
        if s["sinks"] is not None:
            lse = torch.logaddexp(lse, s["sinks"][h * G:(h + 1) * G].double()[None])
    return x.sub_(lse[..., None]).exp_()


def exact(case, seed):
    s = prepare(case, seed)
    block, hkv = case["block"], case["hkv"]
    dev = s["table"].device
    if case["op"] == "select":
        w = _wide(s["w"], block, hkv)[:, 0]
        lens, kept = s["budgets"].clamp(max=s["seq_lens"]), []
        for i in range(case["reqs"]):
            x, n = s["lens"][i], int(lens[i])
            v = w[:, _cells(s, i, dev)]
            at = torch.arange(x, device=dev)
            # the last ones above the first ones above the weights
            last = min(n, case["recent"])
            v = torch.where(at < min(case["first"], n - last), math.inf, v)
            v = torch.where(at >= x - last, math.inf, v)
            order = torch.sort(-v, dim=1, stable=True).indices[:, :n]
            pad = torch.full((hkv, case["keep"] - n), -1, dtype=torch.long, device=dev)
            kept.append(torch.cat([order.sort(1).values, pad], 1).to(torch.int32))
        return torch.stack(kept), lens
    if case["op"] == "compact":
        got = {}
        for name, t in _moved(s).items():
            x = _wide(t, block, hkv)
            for i, n in enumerate(s["keep_each"]):
                c = _cells(s, i, dev)
                for h in range(hkv):
                    x[h][:, c[:n]] = x[h][:, c[s["kept"][i, h, :n].long()]]
            got[name] = x.reshape((t.shape[1], t.shape[0], block) + tuple(t.shape[3:])).transpose(0, 1)
        return got

    def flat(i, h, cache, scale):  # a request's keys or values, [tokens, d]
        b = s["table"][i].long()
        c = (cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache)[:, h][b].double()
        if case["fmt"] != "bf16":
            c = c * (scale[:, h][b].double()[..., None] if case["fmt"] == "token" else scale.double())
        return c.flatten(0, 1)[:s["lens"][i]]

    def gate(i, h):
        if s["g_cache"] is None:
            return None
        G = case["hq"] // hkv
        g = s["g_cache"][s["table"][i].long(), h * G:(h + 1) * G].double()
        return g.transpose(0, 1).flatten(1)[:, :s["lens"][i]]

    if case["op"] == "shared":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        G = case["hq"] // hkv
        for i in range(case["reqs"]):  # each request on its own
            a, r = s["first_row"][i], s["rows"][i]
            for h in range(hkv):
                p = _weights_of(s, i, h, flat(i, h, s["k_cache"], s["k_scale"]), gate(i, h), None)
                out[a:a + r, h * G:(h + 1) * G] = p @ flat(i, h, s["v_cache"], s["v_scale"])
        return out
    w = s["w"].double()
    for i in range(case["reqs"]):
        a, r, n = s["first_row"][i], s["rows"][i], s["lens"][i]
        c = _cells(s, i, dev)
        for h in range(hkv):
            lse = None
            if s["sums"] is not None:
                lse = s["sums"][:, a:a + r].double().unflatten(0, (hkv, -1))[h].T
            new = _weights_of(s, i, h, flat(i, h, s["k_cache"], s["k_scale"]), gate(i, h), lse).sum((0, 1))
            old = w[c // block, h, c % block] * case["decay"]
            old[n - r:] = 0.0
            w[c // block, h, c % block] = new + old
    return w
