"""Measured cases of the operators around the attention calls: the per-head norm with the position
rotation of queries and keys (forward, backward), the write of keys, values and log gates into the
paged cache (plain, or with norm and rotation in the same call) and the read of the cache back into
packed tensors.

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it makes
the library's calls."""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
ROPE_BASE = 10000.0


# ------------------------------------------------------------------------------------------ cases
def _rope(name, op, tokens, hq, hkv, d, rot, interleaved=False, norm=True, max_pos=8192, fused=True):
    """op "fwd" or "bwd"; fused: q and k are views of one projection's output (rows of q, k and v)."""
    return dict(name=name, op=op, tokens=tokens, hq=hq, hkv=hkv, d=d, rot=rot, interleaved=interleaved, norm=norm,
                max_pos=max_pos, fused=fused)


def _append(name, reqs, q_len, ctx, hq, hkv, d, rot, fmt, gates, block, nhd=False, ragged=True):
    """rot > 0: norm and rotation in the same call.  Request i appends up to q_len tokens behind up
    to ctx cached ones; nhd: the cache's slots are outside its heads."""
    return dict(name=name, op="append", reqs=reqs, q_len=q_len, ctx=ctx, hq=hq, hkv=hkv, d=d, rot=rot, fmt=fmt,
                gates=gates, block=block, nhd=nhd, ragged=ragged)


def _gather(name, reqs, ctx, hq, hkv, d, fmt, gates, block, nhd=False, ragged=True):
    return dict(name=name, op="gather", reqs=reqs, q_len=0, ctx=ctx, hq=hq, hkv=hkv, d=d, rot=0, fmt=fmt, gates=gates,
                block=block, nhd=nhd, ragged=ragged)


def listed():
    return [
        # one decoding step of 64 requests, positions up to 32768: latency
        _rope("rope_fwd_decode_64", "fwd", 64, 64, 4, 128, 128, max_pos=32768),
        # a training step's packed 8192 tokens, GQA 32 / 8
        _rope("rope_fwd_8192_d128", "fwd", 8192, 32, 8, 128, 128),
        # the widest heads, a quarter of the dims rotated in neighbouring pairs
        _rope("rope_fwd_16384_d512", "fwd", 16384, 32, 4, 512, 128, interleaved=True, max_pos=16384, fused=False),
        # a short sequence of small heads
        _rope("rope_bwd_129_d64", "bwd", 129, 2, 2, 64, 64, max_pos=256),
        # the training step's backward
        _rope("rope_bwd_8192_d128", "bwd", 8192, 32, 8, 128, 128),
        # wide heads, half of the dims rotated
        _rope("rope_bwd_8191_d256", "bwd", 8191, 16, 4, 256, 128, interleaved=True, fused=False),
        # one decoding step: norm, rotation and write of 64 single tokens, with gates
        _append("append_rope_decode_64x1", 64, 1, 4096, 64, 4, 128, 128, "token", True, 16),
        # a chunked prefill's write: four chunks of 1024 tokens with the norm and the rotation
        _append("append_rope_chunk_4x1024", 4, 1024, 32768, 64, 4, 128, 128, "token", False, 16, ragged=False),
        # long prompts with gates, keys made elsewhere
        _append("append_prompt_4x16384", 4, 16384, 1, 32, 8, 128, 0, "token", True, 64, nhd=True),
        # a bf16 cache with wide heads
        _append("append_bf16_8x512_d256", 8, 512, 2048, 16, 4, 256, 0, "bf16", False, 32),
        # a few short contexts read back
        _gather("gather_3x300", 3, 300, 16, 1, 128, "token", True, 16),
        # the contexts of a chunked prefill read back
        _gather("gather_4x32768", 4, 32768, 64, 4, 128, "token", False, 16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        d = rng.choice([64, 128, 128, 128, 256, 512])
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 7, 8, 16])
        rot = rng.choice([d, d, d // 2, d // 4])
        op = rng.choice(["fwd", "bwd", "append", "append", "gather"])
        if op in ("fwd", "bwd"):
            c = _rope("", op, _log_int(rng, 1, 16384), hq, hkv, d, rot, rng.random() < 0.4, rng.random() < 0.8,
                      _log_int(rng, 64, 65536), rng.random() < 0.5)
        else:
            fmt = rng.choice(["token", "token", "tensor", "bf16"])
            reqs, block = _log_int(rng, 1, 64), rng.choice([16, 32, 64, 128])
            gates, nhd = rng.random() < 0.5, rng.random() < 0.5
            if op == "append":
                c = _append("", reqs, _log_int(rng, 1, 8192), _log_int(rng, 1, 8192), hq, hkv, d,
                            rot if rng.random() < 0.5 else 0, fmt, gates, block, nhd)
            else:
                c = _gather("", reqs, _log_int(rng, 1, 32768), hq, hkv, d, fmt, gates, block, nhd)
        del c["name"]
        # the cache and, with gates, its cumulative gates stay within a few GB
        if op in ("append", "gather") and c["reqs"] * (c["ctx"] + c["q_len"]) * (hkv * d * 2 + hq) > 1 << 30:
            continue
        if work(c)["bytes"] <= most:
            return c


# ----------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """(appended or read rows, cached tokens) of each request, from the case alone."""
    rows, ctx = [], []
    for i in range(case["reqs"]):
        f = ((i * 7 + 3) % 11 + 1) / 11.0 if case["ragged"] else 1.0
        g = ((i * 5 + 4) % 13 + 1) / 13.0 if case["ragged"] else (i + 1) / case["reqs"]
        if case["op"] == "gather":
            n = max(1, int(case["ctx"] * g))
            rows.append(n)
            ctx.append(n)
        else:
            n = max(1, int(case["q_len"] * f))
            rows.append(n)
            # ctx 1: prompts with nothing before them
            ctx.append(n if case["ctx"] == 1 else n + int((case["ctx"] - 1) * g))
    return rows, ctx


def _table(max_pos, rot, dev):
    """fp32 [max_pos, rot]: the cosines, then the sines, of position * base^(-2 i / rot)."""
    freq = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _heads(gen, tokens, heads, d, dev):
    """A projection's output: tokens and heads of different sizes, some dims larger than others."""
    x = torch.randn((tokens, heads, d), generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn((tokens, heads, 1), generator=gen, device=dev))
    x *= torch.exp(0.5 * torch.randn((1, heads, d), generator=gen, device=dev))
    return x


def _qkv(gen, case, tokens, dev, fused):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    x = _heads(gen, tokens, hq + 2 * hkv, d, dev).to(torch.bfloat16)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def _weights(gen, d, dev):
    return [1.0 + 0.2 * torch.randn(d, generator=gen, device=dev) for _ in range(2)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] in ("fwd", "bwd"):
        n = case["tokens"]
        s["q"], s["k"], _ = _qkv(gen, case, n, dev, case["fused"])
        s["qw"], s["kw"] = _weights(gen, d, dev) if case["norm"] else (None, None)
        s["table"] = _table(case["max_pos"], case["rot"], dev)
        s["pos"] = torch.randint(0, case["max_pos"], (n,), generator=gen, device=dev, dtype=torch.int32)
        if case["op"] == "bwd":
            s["dq"] = _heads(gen, n, hq, d, dev).to(torch.bfloat16)
            s["dk"] = _heads(gen, n, hkv, d, dev).to(torch.bfloat16)
        return s
    rows, ctx = _lengths(case)
    block = case["block"]
    pages = [-(-n // block) for n in ctx]
    nb = sum(pages) + 8
    perm = torch.randperm(nb, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((case["reqs"], max(pages)), dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = perm[at:at + n]
        at += n
    s["block_table"] = table
    s["seq_lens"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    cu = [0]
    for n in rows:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["total"], s["longest"] = cu[-1], max(rows)

    def cache():
        shape = (nb, block, hkv, d) if case["nhd"] else (nb, hkv, block, d)
        x = torch.randn(shape, generator=gen, device=dev)
        if case["fmt"] == "bf16":
            x = x.to(torch.bfloat16)
        else:
            x = (x * 100.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        return x.permute(0, 2, 1, 3) if case["nhd"] else x

    def scale():
        if case["fmt"] == "token":  # of earlier rows: a spread of twenty
            return torch.exp(torch.rand((nb, hkv, block), generator=gen, device=dev) * math.log(20.0)) / 64.0
        if case["fmt"] == "tensor":  # one for the whole cache, from a calibration
            return torch.rand((1,), generator=gen, device=dev) * 0.05 + 0.02
        return None

    s["k_cache"], s["v_cache"] = cache(), cache()
    s["k_scale"], s["v_scale"] = scale(), scale()
    s["g_cache"] = None
    if case["gates"]:
        # cumulative gates of a context: about -0.05 a token
        s["g_cache"] = -200.0 * torch.rand((nb, hq, block), generator=gen, device=dev)
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = _qkv(gen, case, s["total"], dev, case["rot"] > 0)
        s["log_gate"] = None
        if case["gates"]:
            z = 3.0 + torch.randn((s["total"], hq), generator=gen, device=dev)
            s["log_gate"] = -torch.log1p(torch.exp(-z))
        if case["rot"]:
            s["qw"], s["kw"] = _weights(gen, d, dev)
            s["table"] = _table(max(ctx), case["rot"], dev)
    return s


# ------------------------------------------------------------------------------------- plain forms
def _turn(x, rows, rot, interleaved, back=False):
    """Rotates the first rot dims of x [tokens, heads, d] by the table's rows [tokens, rot]."""
    c, s = rows[:, None, :rot // 2], rows[:, None, rot // 2:]
    s = -s if back else s
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _norm_turn(x, w, rows, rot, interleaved, norm):
    x = x.float()
    if norm:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return _turn(x, rows, rot, interleaved)


def _norm_turn_back(dy, x, w, rows, rot, interleaved, norm):
    g = _turn(dy.float(), rows, rot, interleaved, back=True)
    if not norm:
        return g.to(torch.bfloat16), None
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    dw = (g * n).sum((0, 1), dtype=torch.float64).float()
    u = g * w
    return (r * (u - n * (u * n).mean(-1, keepdim=True))).to(torch.bfloat16), dw


def _places(s):
    """(request, position, block, slot) of every packed row."""
    t = torch.arange(s["total"], device=s["cu"].device, dtype=torch.int32)
    r = torch.searchsorted(s["cu"], t, right=True) - 1
    pos = s["seq_lens"][r] - s["cu"][r + 1] + t
    return r, pos, s["block_table"][r, (pos // s["block"]).long()].long(), (pos % s["block"]).long()


def _before(s, r, pos):
    """The cumulative gates of the position before `pos`: 0 before the first."""
    p = (pos - 1).clamp(min=0)
    g = s["g_cache"][s["block_table"][r, (p // s["block"]).long()].long(), :, (p % s["block"]).long()]
    return torch.where(pos[:, None] > 0, g, torch.zeros_like(g))


def _write(x, cache, scale, fmt, block, slot):
    if fmt == "bf16":
        cache[block, :, slot] = x.to(torch.bfloat16)
        return
    x = x.float()
    if fmt == "token":
        sc = x.abs().amax(-1) / E4M3_MAX
        scale[block, :, slot] = sc
        sc = sc[..., None]
    else:
        sc = scale
    y = torch.where(sc > 0, x / sc, torch.zeros_like(x)).clamp(-E4M3_MAX, E4M3_MAX)
    cache[block, :, slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)


def _append_plain(s):
    r, pos, block, slot = _places(s)
    k, q = s["k"], None
    if s["rot"]:
        rows = s["table"][pos.long()]
        q = _norm_turn(s["q"], s["qw"], rows, s["rot"], False, True).to(torch.bfloat16)
        k = _norm_turn(k, s["kw"], rows, s["rot"], False, True)
    if s["log_gate"] is not None:
        c = s["log_gate"].cumsum(0, dtype=torch.float64)
        first = s["cu"][r].long()
        c = c - c[first] + s["log_gate"][first]
        prev = _before(s, r, s["seq_lens"][r] - s["cu"][r + 1] + s["cu"][r])
        s["g_cache"][block, :, slot] = (prev + c).float()
    _write(k, s["k_cache"], s["k_scale"], s["fmt"], block, slot)
    _write(s["v"], s["v_cache"], s["v_scale"], s["fmt"], block, slot)
    return q


def _read(cache, scale, fmt, block, slot):
    x = cache[block, :, slot]
    if fmt == "bf16":
        return x
    x = x.view(torch.float8_e4m3fn).float()
    return (x * (scale[block, :, slot][..., None] if fmt == "token" else scale)).to(torch.bfloat16)


def _gather_plain(s):
    r, pos, block, slot = _places(s)
    gate = None
    if s["g_cache"] is not None:
        gate = s["g_cache"][block, :, slot] - _before(s, r, pos)
    return (_read(s["k_cache"], s["k_scale"], s["fmt"], block, slot),
            _read(s["v_cache"], s["v_scale"], s["fmt"], block, slot), gate)


def _held(cache, fmt):
    return cache if fmt == "bf16" else cache.view(torch.float8_e4m3fn)


def run(s):
    if own:
        import gated_causal_softmax_gb300 as gcs
    if s["op"] == "fwd":
        if own:
            return gcs.attn_qk_norm_rope_fwd(s["q"], s["k"], s["table"], s["pos"], s["qw"], s["kw"], EPS,
                                             norm=s["norm"], interleaved=s["interleaved"])
        rows = s["table"][s["pos"].long()]
        return tuple(_norm_turn(x, w, rows, s["rot"], s["interleaved"], s["norm"]).to(torch.bfloat16)
                     for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
    if s["op"] == "bwd":
        if own:
            return gcs.attn_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["table"], s["pos"], s["qw"], s["kw"],
                                             EPS, norm=s["norm"], interleaved=s["interleaved"])
        rows = s["table"][s["pos"].long()]
        dq, dqw = _norm_turn_back(s["dq"], s["q"], s["qw"], rows, s["rot"], s["interleaved"], s["norm"])
        dk, dkw = _norm_turn_back(s["dk"], s["k"], s["kw"], rows, s["rot"], s["interleaved"], s["norm"])
        return dq, dk, dqw, dkw
    if s["op"] == "gather":
        if own:
            return gcs.attn_cache_gather(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                         s["seq_lens"], s["cu"], s["total"], g_cache=s["g_cache"])
        return _gather_plain(s)
    if own and s["rot"]:
        q = gcs.attn_cache_append_rope(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                       s["block_table"], s["seq_lens"], s["cu"], s["longest"], s["table"], None,
                                       s["qw"], s["kw"], EPS, log_gate=s["log_gate"], g_cache=s["g_cache"])
    elif own:
        q = gcs.attn_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                  s["block_table"], s["seq_lens"], s["cu"], s["longest"], log_gate=s["log_gate"],
                                  g_cache=s["g_cache"])
    else:
        q = _append_plain(s)
    token = s["fmt"] == "token"
    return {"q": q, "k": _held(s["k_cache"], s["fmt"]), "v": _held(s["v_cache"], s["fmt"]), "g": s["g_cache"],
            "k_scale": s["k_scale"] if token else None, "v_scale": s["v_scale"] if token else None}


# ------------------------------------------------------------------------------------------- work
def work(case):
    hq, hkv, d, rot = case["hq"], case["hkv"], case["d"], case["rot"]
    if case["op"] in ("fwd", "bwd"):
        n, norm = case["tokens"], case["norm"]
        e = n * (hq + hkv) * d
        b = 4 * n + 4 * rot * min(n, case["max_pos"])  # positions and the table's rows
        if case["op"] == "fwd":
            return {"bytes": b + 4 * e + 8 * d * norm, "flops": 7 * e if norm else 3 * n * (hq + hkv) * rot}
        # without a norm the gradient does not depend on q and k
        return {"bytes": b + (6 * e + 16 * d if norm else 4 * e), "flops": 14 * e if norm else 3 * n * (hq + hkv) * rot}
    rows, ctx = _lengths(case)
    n = sum(rows)
    held = 2 if case["fmt"] == "bf16" else 1
    e = 2 * n * hkv * d
    b = e * (2 + held) + (8 * n * hkv if case["fmt"] == "token" else 0) + 8 * case["reqs"] + 4 * (n // case["block"])
    b += 8 * n * hq if case["gates"] else 0
    f = (4 if case["op"] == "append" else 1) * e + (n * hq if case["gates"] else 0)
    if rot:
        b += 4 * n * hq * d + 4 * rot * min(n, max(ctx)) + 8 * d
        f += 7 * n * (hq + hkv) * d
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------- values in 64 bits
def _angles(case, pos, rot):
    """The table's entries are inputs: its rows, widened."""
    c = _table(case["max_pos"] if "max_pos" in case else int(pos.max()) + 1, rot, pos.device)[pos.long()].double()
    return torch.complex(c[:, :rot // 2], c[:, rot // 2:])[:, None]


def _spin(x, z, rot, interleaved):
    """The rotation as a product of complex numbers."""
    m = rot // 2
    if interleaved:
        p = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], m, 2).contiguous()) * z
        y = torch.view_as_real(p).flatten(-2)
    else:
        p = torch.complex(x[..., :m].contiguous(), x[..., m:rot].contiguous()) * z
        y = torch.cat([p.real, p.imag], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _exact_fwd(x, w, z, rot, interleaved):
    x = x.double()
    if w is not None:
        x = w.double() * x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return _spin(x, z, rot, interleaved)


def _exact_bwd(dy, x, w, z, rot, interleaved):
    g = _spin(dy.double(), z.conj(), rot, interleaved)
    if w is None:
        return g, None
    x, d = x.double(), x.shape[-1]
    ms = x.square().sum(-1, keepdim=True) / d + EPS
    gw = g * w.double()
    # d(x ms^-1/2) = dx ms^-1/2 - x ms^-3/2 (x . dx) / d
    dx = gw / ms.sqrt() - x * ((gw * x).sum(-1, keepdim=True) / (d * ms * ms.sqrt()))
    return dx, torch.einsum("thd,thd->d", g, x / ms.sqrt())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        z = _angles(case, s["pos"], case["rot"])
        if case["op"] == "fwd":
            return tuple(_exact_fwd(x, w, z, case["rot"], case["interleaved"])
                         for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])))
        dq, dqw = _exact_bwd(s["dq"], s["q"], s["qw"], z, case["rot"], case["interleaved"])
        dk, dkw = _exact_bwd(s["dk"], s["k"], s["kw"], z, case["rot"], case["interleaved"])
        return dq, dk, dqw, dkw
    rows, ctx = _lengths(case)
    dev, block, fmt = s["cu"].device, case["block"], case["fmt"]
    parts = [(i, torch.arange(ctx[i] - rows[i], ctx[i], device=dev)) for i in range(case["reqs"])]
    blk = torch.cat([s["block_table"][i][p // block] for i, p in parts]).long()
    pos = torch.cat([p for _, p in parts])
    cell = blk * block + pos % block

    def flat(t):  # [blocks, heads, slots, ...] -> a copy [blocks * slots, heads, ...] in 64 bits
        if t.dtype == torch.uint8:
            t = t.view(torch.float8_e4m3fn)
        return t.transpose(1, 2).flatten(0, 1).double()

    def back(t):  # and back
        return t.unflatten(0, (-1, block)).transpose(1, 2)

    if case["op"] == "gather":
        out = []
        for c, sc in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
            x = flat(c)[cell]
            out.append(x if fmt == "bf16" else x * (flat(sc)[cell][..., None] if fmt == "token" else sc.double()))
        gate = None
        if s["g_cache"] is not None:
            g, at = flat(s["g_cache"])[cell], 0
            gate = g.clone()
            for n in rows:  # the whole context is read: the first row has nothing before it
                gate[at + 1:at + n] -= g[at:at + n - 1]
                at += n
        return out[0], out[1], gate
    got = dict(q=None, k=None, v=None, g=None, k_scale=None, v_scale=None)
    new = dict(k=s["k"].double(), v=s["v"].double())
    if case["rot"]:
        z = _angles(case, pos, case["rot"])
        got["q"] = _exact_fwd(s["q"], s["qw"], z, case["rot"], False)
        new["k"] = _exact_fwd(s["k"], s["kw"], z, case["rot"], False)
    for name in ("k", "v"):
        x, held = new[name], flat(s[name + "_cache"])
        if fmt == "token":
            sc, scales = x.abs().amax(-1) / E4M3_MAX, flat(s[name + "_scale"])
            scales[cell] = sc
            got[name + "_scale"] = back(scales)
            x = x / sc[..., None]  # what the codes stand for, before their rounding
        elif fmt == "tensor":
            x = (x / s[name + "_scale"].double()).clamp(-E4M3_MAX, E4M3_MAX)
        held[cell] = x
        got[name] = back(held)
    if s["g_cache"] is not None:
        g, at = flat(s["g_cache"]), 0
        for (i, p), n in zip(parts, rows):
            c = s["log_gate"][at:at + n].double().cumsum(0)
            if int(p[0]) > 0:
                q = int(p[0]) - 1
                c = c + g[int(s["block_table"][i, q // block]) * block + q % block]
            g[cell[at:at + n]] = c
            at += n
        got["g"] = back(g)
    return got
