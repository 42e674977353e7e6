"""Cases of the calls that a serving loop makes around the paged decode step.

Four operators: the append with rotary positions of several axes (rope), the accumulated attention weight of
every cached token (weights), the eviction of a cache by that weight (evict), and the verification of drafted
tokens (verify).  ``run`` computes their plain forms from elementary torch operations, or, where ``own`` is
true, calls the library, bound once as a serving loop binds its calls (``ops.prepare``).
"""
import math

import numpy as np
import torch

own = False

BS = 16
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the four sequences of the tiny batch at decode: launch latency
        dict(name="rope_4_tokens", op="rope", T=4, Hq=8, Hkv=2, D=64, dtype="f16", pool="16", axes=1,
             rotary=64, adjacent=False),
        # 128 sequences with 4 drafted tokens each, three axes
        dict(name="rope_512_drafts", op="rope", T=512, Hq=28, Hkv=4, D=128, dtype="f16", pool="16", axes=3,
             rotary=128, adjacent=False),
        # a long prompt with an image in it, adjacent pairs, partly rotated heads
        dict(name="rope_prompt_16k", op="rope", T=16384, Hq=28, Hkv=4, D=128, dtype="bf16", pool="16", axes=3,
             rotary=96, adjacent=True),
        # the tiny batch: the smallest call
        dict(name="weights_tiny", op="weights", B=4, Hq=8, Hkv=2, D=64, dtype="f16", pool="16", lo=1, hi=256,
             lens="uniform", n_q=1, decay=1.0),
        # one decode step of a 128-sequence batch, 28/4 heads
        dict(name="weights_batch_128", op="weights", B=128, Hq=28, Hkv=4, D=128, dtype="f16", pool="16", lo=1,
             hi=8192, lens="lognormal", n_q=1, decay=0.875),
        # two long contexts in E4M3, scored by the prompt's last 4 tokens
        dict(name="weights_long_e4m3", op="weights", B=2, Hq=28, Hkv=4, D=128, dtype="bf16", pool="fp8",
             lo=100000, hi=131072, lens="uniform", n_q=4, decay=0.0),
        # a small cache cut to a quarter
        dict(name="evict_tiny", op="evict", B=4, Hkv=2, D=64, pool="16", lo=65, hi=256, keep=64, first=4,
             recent=16),
        # 48 sequences past their budget, each cut to 1024 tokens
        dict(name="evict_batch_48", op="evict", B=48, Hkv=2, D=128, pool="16", lo=1100, hi=4096, keep=1024,
             first=4, recent=256),
        # long E4M3 prompts cut to a fixed cache, an odd budget
        dict(name="evict_long_e4m3", op="evict", B=8, Hkv=4, D=128, pool="fp8", lo=20000, hi=32768, keep=4099,
             first=16, recent=1000),
        # one sequence, four drafts, a small vocabulary: latency
        dict(name="verify_one", op="verify", B=1, n=4, V=32000, dtype="f32", draft="probs", agree=0.7),
        # a batch of 128 with three drafts each
        dict(name="verify_batch_128", op="verify", B=128, n=3, V=128000, dtype="f32", draft="probs", agree=0.8),
        # drafts without probabilities (looked up in the prompt), bf16 target, odd vocabulary
        dict(name="verify_lookup", op="verify", B=33, n=7, V=50257, dtype="bf16", draft="none", agree=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "weights", "evict", "verify"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    pool = rng.choice(["16", "16", "fp8"])
    if op == "rope":
        T = _log(rng, 1, 14000) if pool == "16" else _log(rng, 1, 2000)
        Hkv, G = min(Hkv, 4), min(G, 7)
        return dict(op=op, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["f16", "bf16"]), pool=pool,
                    axes=rng.choice([1, 2, 3]), rotary=rng.choice([32, D // 2, D]),
                    adjacent=rng.random() < 0.5)
    if op == "weights":
        n_q = rng.choice([1, 1, 2, 4])
        budget = 300000 // Hkv   # tokens in all
        hi = _log(rng, 16, min(40000, budget))
        B = max(1, min(_log(rng, 1, 100), budget // hi))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["f16", "bf16"]), pool=pool,
                    lo=rng.randint(1, hi), hi=hi, lens="uniform", n_q=n_q, decay=rng.choice([0.0, 0.5, 1.0]))
    if op == "evict":
        budget = 300000 // Hkv
        hi = _log(rng, 40, 30000)
        B = max(1, min(_log(rng, 1, 64), budget // hi))
        keep = rng.randint(8, max(8, hi // 2))
        return dict(op=op, B=B, Hkv=Hkv, D=D, pool=pool, lo=rng.randint(1, hi), hi=hi, keep=keep,
                    first=rng.randint(0, min(8, keep // 2)), recent=rng.randint(0, keep // 2))
    V = _log(rng, 500, 130000)
    n = rng.randint(1, 8)
    B = max(1, min(_log(rng, 1, 128), 50_000_000 // (V * (n + 1))))
    return dict(op=op, B=B, n=n, V=V, dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                draft=rng.choice(["probs", "probs", "none"]), agree=round(rng.uniform(0.2, 0.95), 3))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    out = torch.empty(shape, device="cuda", dtype=dtype)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        n = min(1 << 26, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").to(dtype)
    return out


def _lens(case, g):
    if case["lens"] == "lognormal":
        z = torch.randn(case["B"], generator=g, device="cuda", dtype=torch.float64)
        L = torch.exp(math.log(1024) + z).round()
    else:
        z = torch.rand(case["B"], generator=g, device="cuda", dtype=torch.float64)
        L = (case["lo"] + z * (case["hi"] - case["lo"] + 1)).floor()
    return L.clamp(case["lo"], case["hi"]).to(torch.int32)


def _tables(L, mbs, g):
    """A shuffled pool of as many blocks as the sequences need, and their tables (-1 past each one's blocks)."""
    nb = (L.long() + BS - 1) // BS
    total = int(nb.sum())
    used = torch.arange(mbs, device="cuda")[None, :] < nb[:, None]
    t = torch.full((L.numel(), mbs), -1, dtype=torch.int32, device="cuda")
    t[used] = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    return t, total


def _e4m3_pool(g, nb, Hkv, D):
    """Codes and page scales of pages whose values are of order one."""
    codes = torch.empty(nb, Hkv, BS, D, dtype=torch.uint8, device="cuda")
    scale = torch.empty(nb, Hkv, dtype=torch.float32, device="cuda")
    for i in range(0, nb, 4096):
        x = torch.randn(min(4096, nb - i), Hkv, BS, D, generator=g, device="cuda")
        s = x.abs().amax(dim=(2, 3)) / 448
        codes[i:i + 4096] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[i:i + 4096] = s
    return codes, scale


def _spec(case):
    half = case["rotary"] // 2
    i = np.arange(half, dtype=np.float64)
    inv_freq = 1e6 ** (-i / half)
    # contiguous sections: the first quarter of the pairs turns with the first axis, the rest in equal parts
    axes = case["axes"]
    cut = [0, half] if axes == 1 else [0, half // 4] + [half // 4 + (half - half // 4) * k // (axes - 1)
                                                       for k in range(1, axes)]
    axis = np.zeros(half, dtype=np.int32)
    for a in range(axes):
        axis[cut[a]:cut[a + 1]] = a
    return inv_freq, axis


def _inputs(case, seed):
    return {"rope": _prepare_rope, "weights": _prepare_weights, "evict": _prepare_evict,
            "verify": _prepare_verify}[case["op"]](case, _gen(seed))


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if own:
        s["call"] = _bind(case, s)
    return s


def _prepare_rope(case, g):
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    dt = DT[case["dtype"]]
    qkv = _randn(g, (T, (Hq + 2 * Hkv) * D), dt)        # one projection's output: q, k and v are views of it
    nb = T if case["pool"] == "fp8" else (T + BS - 1) // BS + 8
    start = int(torch.randint(0, 60000, (1,), generator=g, device="cuda"))
    i = torch.arange(T, device="cuda", dtype=torch.int32)
    pos = (start + i)[None].repeat(case["axes"], 1)
    if case["axes"] > 1:                                # an image in the middle: its rows and columns
        w = max(1, math.isqrt(T // 2))
        img = (i >= T // 4) & (i < T // 4 + T // 2)
        k = i - T // 4
        for a, step in enumerate([torch.zeros_like(k), k // w, k % w][:case["axes"]]):
            pos[a] = torch.where(img, start + T // 4 + step, pos[a])
    inv_freq, axis = _spec(case)
    s = {"q": qkv[:, :Hq * D].view(T, Hq, D), "k": qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
         "v": qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D), "pos": pos.contiguous(), "inv_freq": inv_freq,
         "axis": axis, "q_out": torch.zeros(T, Hq, D, dtype=dt, device="cuda")}
    if case["pool"] == "fp8":                           # one token of each page, its first
        s["slots"] = torch.randperm(nb, generator=g, device="cuda")[:T] * BS
        for n in "kv":
            s[n + "c"] = torch.zeros(nb, Hkv, BS, D, dtype=torch.uint8, device="cuda")
            s[n + "s"] = torch.ones(nb, Hkv, dtype=torch.float32, device="cuda")
    else:
        s["slots"] = torch.randperm(nb * BS, generator=g, device="cuda")[:T]
        for n in "kv":
            s[n + "c"] = torch.zeros(nb, Hkv, BS, D, dtype=dt, device="cuda")
    return s


def _prepare_weights(case, g):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    dt = DT[case["dtype"]]
    L = _lens(case, g)
    mbs = (case["hi"] + BS - 1) // BS
    bt, nb = _tables(L, mbs, g)
    s = {"lens": L, "bt": bt, "scale": float(np.float32(1 / math.sqrt(D)))}
    shape = (B, Hq, D) if case["n_q"] == 1 else (B, case["n_q"], Hq, D)
    s["q"] = _randn(g, shape, dt) * 2                   # some tokens get far more weight than others
    if case["pool"] == "fp8":
        s["kc"], s["ks"] = _e4m3_pool(g, nb, Hkv, D)
    else:
        s["kc"] = _randn(g, (nb, Hkv, BS, D), dt)
    live = torch.arange(mbs * BS, device="cuda")[None, None] < L[:, None, None]
    s["w"] = torch.rand(B, Hkv, mbs * BS, generator=g, device="cuda") * live
    return s


def _prepare_evict(case, g):
    B, Hkv, D, keep = case["B"], case["Hkv"], case["D"], case["keep"]
    L = _lens({**case, "lens": "uniform"}, g)
    mbs = (case["hi"] + BS - 1) // BS
    bt, nb = _tables(L, mbs, g)
    kb = (keep + BS - 1) // BS
    spare = nb + torch.randperm(B * kb, generator=g, device="cuda").to(torch.int32).view(B, kb)
    s = {"lens": L, "bt": bt, "spare": spare, "nb": nb}
    for n in "kv":
        if case["pool"] == "fp8":
            codes, scale = _e4m3_pool(g, nb, Hkv, D)
            s[n + "c"] = torch.cat([codes, torch.zeros(B * kb, Hkv, BS, D, dtype=torch.uint8, device="cuda")])
            s[n + "s"] = torch.cat([scale, torch.ones(B * kb, Hkv, device="cuda")])
        else:
            s[n + "c"] = torch.cat([_randn(g, (nb, Hkv, BS, D), torch.float16),
                                    torch.zeros(B * kb, Hkv, BS, D, dtype=torch.float16, device="cuda")])
    # accumulated weights: a few heavy tokens, many light ones, some that nothing ever looked at
    w = torch.randn(B, Hkv, mbs * BS, generator=g, device="cuda").mul_(2).exp_()
    s["w"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
    s["w_out"] = torch.zeros(B, Hkv, kb * BS, device="cuda")
    s["kept"] = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["bt_out"] = torch.full((B, kb), -1, dtype=torch.int32, device="cuda")
    return s


def _prepare_verify(case, g):
    B, n, V = case["B"], case["n"], case["V"]
    dt = {"f32": torch.float32, **DT}[case["dtype"]]
    logits = torch.randn(B, n + 1, V, generator=g, device="cuda") * 3
    p = torch.softmax(logits, -1)
    s = {"q": None}
    if case["draft"] == "probs":                        # the draft model: the target's logits, blurred
        noise = torch.randn(B, n, V, generator=g, device="cuda")
        a = case["agree"]
        q = torch.softmax(logits[:, :n] * a + noise * (1 - a) * 3, -1)
        s["q"] = q.to(dt)
        at = q
    else:
        at = p[:, :n]
    u = torch.rand(B, n, 1, generator=g, device="cuda", dtype=torch.float64)
    cdf = at.double().cumsum(-1)
    s["x"] = (cdf <= u * cdf[..., -1:]).sum(-1).clamp(max=V - 1).to(torch.int32)
    s["p"] = p.to(dt)
    s["u"] = torch.rand(B, n + 1, generator=g, device="cuda")
    s["drafts"] = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    s["drafts"][::2] = n                                # half of the sequences have them all
    s["out"] = torch.full((B, n + 1), -1, dtype=torch.int32, device="cuda")
    s["acc"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------- the library's calls
def _bind_rope(case, s):
    from paged_kv_cache_179_gb300 import ops
    spec = ops.RopeSpec(s["inv_freq"], s["axis"], adjacent=case["adjacent"])
    if case["pool"] == "fp8":
        return ops.prepare(lambda: ops.pa_rope_append_fp8(
            s["q_out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["slots"], s["pos"], spec))
    return ops.prepare(lambda: ops.pa_rope_append(
        s["q_out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["pos"], spec))


def _bind_weights(case, s):
    from paged_kv_cache_179_gb300 import ops
    s["ws"] = ops.alloc_weights_workspace(case["B"], case["Hq"], case["Hkv"], case["hi"], case["n_q"],
                                          s["q"].device)
    args = (s["bt"], s["lens"], case["hi"], s["scale"], s["ws"])
    if case["pool"] == "fp8":
        return ops.prepare(lambda: ops.pa_attention_weights_fp8(
            s["w"], s["q"], s["kc"], s["ks"], *args, decay=case["decay"], fresh_tokens=case["n_q"]))
    return ops.prepare(lambda: ops.pa_attention_weights(
        s["w"], s["q"], s["kc"], *args, decay=case["decay"], fresh_tokens=case["n_q"]))


def _bind_evict(case, s):
    from paged_kv_cache_179_gb300 import ops
    args = (s["w"], s["w_out"], s["bt"], s["lens"], case["hi"], s["spare"], s["bt_out"], s["new_lens"], s["kept"])
    kw = dict(first_tokens=case["first"], recent_tokens=case["recent"])
    if case["pool"] == "fp8":
        return ops.prepare(lambda: ops.pa_evict_fp8(s["kc"], s["vc"], s["ks"], s["vs"], *args, **kw))
    return ops.prepare(lambda: ops.pa_evict(s["kc"], s["vc"], *args, **kw))


def _bind_verify(case, s):
    from paged_kv_cache_179_gb300 import ops
    return ops.prepare(lambda: ops.pa_verify_drafts(s["out"], s["acc"], s["p"], s["q"], s["x"], s["u"],
                                                    num_drafts=s["drafts"]))


def _bind(case, s):
    return {"rope": _bind_rope, "weights": _bind_weights, "evict": _bind_evict,
            "verify": _bind_verify}[case["op"]](case, s)


# ------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        s["call"]()
    else:
        {"rope": _plain_rope, "weights": _plain_weights, "evict": _plain_evict,
         "verify": _plain_verify}[case["op"]](case, s)
    return _outputs(case, s)


def _outputs(case, s):
    fp8 = case.get("pool") == "fp8"
    if case["op"] == "rope":
        # E4M3 codes as the values they stand for, in units of their page's scale
        kv = {n: s[n].view(torch.float8_e4m3fn) if fp8 else s[n] for n in ("kc", "vc")}
        return {"q": s["q_out"], **kv, **({"ks": s["ks"], "vs": s["vs"]} if fp8 else {})}
    if case["op"] == "weights":
        return {"w": s["w"]}
    if case["op"] == "evict":
        nb = s["nb"]                                    # the spare blocks are behind the sources in the pool
        kv = {n: s[n][nb:].view(torch.float8_e4m3fn) if fp8 else s[n][nb:] for n in ("kc", "vc")}
        more = {"ks": s["ks"][nb:], "vs": s["vs"][nb:]} if fp8 else {}
        return {**kv, **more, "w": s["w_out"], "kept": s["kept"], "lens": s["new_lens"], "tables": s["bt_out"]}
    return {"tokens": s["out"], "accepted": s["acc"]}


def _turn(x, cos, sin, rotary, adjacent):
    """x [T][H][D] rotated in 32 bits by the angles whose cos and sin are [T][rotary / 2]."""
    x = x.float()
    r, rest = x[..., :rotary], x[..., rotary:]
    c, s = cos[:, None], sin[:, None]
    if adjacent:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r.chunk(2, -1)
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def _page_scale(amax):
    """amax / 448 (a tensor divided by a tensor: by a number, it would be multiplied with the reciprocal)."""
    return torch.where(amax > 0, amax / torch.full_like(amax, 448), torch.ones_like(amax))


def _plain_rope(case, s):
    angle = (s["pos"].double()[torch.from_numpy(s["axis"]).to("cuda").long()]      # 64 bits: positions far out
             * torch.from_numpy(s["inv_freq"]).to("cuda")[:, None]).T
    cos, sin = angle.cos().float(), angle.sin().float()
    s["q_out"].copy_(_turn(s["q"], cos, sin, case["rotary"], case["adjacent"]))
    k = _turn(s["k"], cos, sin, case["rotary"], case["adjacent"]).to(s["q"].dtype)
    blk, row = s["slots"] // BS, s["slots"] % BS
    if case["pool"] == "fp8":                           # each row opens its page: scale amax / 448
        for n, x in (("k", k.float()), ("v", s["v"].float())):
            sc = _page_scale(x.abs().amax(-1))
            s[n + "s"][blk] = sc
            s[n + "c"][blk, :, row] = (x / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["kc"][blk, :, row] = k
        s["vc"][blk, :, row] = s["v"]


def _plain_weights(case, s):
    B, Hkv, D, n_q = case["B"], case["Hkv"], case["D"], case["n_q"]
    G = case["Hq"] // Hkv
    bt = s["bt"].clamp(min=0).long()
    n = bt.shape[1] * BS
    k = s["kc"][bt]                                     # [B][blocks][Hkv][16][D]
    if case["pool"] == "fp8":
        k = k.view(torch.float8_e4m3fn).float() * s["ks"][bt][..., None, None]
    k = k.float().transpose(1, 2).reshape(B, Hkv, n, D)
    q = s["q"].float().view(B, n_q, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n_q * G, D)
    x = q @ k.transpose(-1, -2) * s["scale"]            # [B][Hkv][n_q * G][n]
    t = torch.arange(n, device="cuda")
    end = s["lens"][:, None] - n_q + 1 + torch.arange(n_q, device="cuda").repeat_interleave(G)   # [B][rows]
    x = x.masked_fill(t >= end[:, None, :, None], -math.inf)
    e = (x - x.amax(-1, keepdim=True).clamp(min=-3e38)).exp()
    p = (e / e.sum(-1, keepdim=True).clamp(min=1e-30)).sum(2)
    L = s["lens"][:, None, None]
    old = torch.where(t < L - n_q, s["w"] * case["decay"], torch.zeros_like(s["w"]))
    s["w"].copy_(torch.where(t < L, old + p, s["w"]))


def _plain_evict(case, s):
    B, Hkv, keep = case["B"], case["Hkv"], case["keep"]
    n = s["w"].shape[-1]
    t = torch.arange(n, device="cuda")
    L = s["lens"].long()[:, None, None]
    # the places in the order in which they are kept: protected ones, then by weight, the lowest index first
    key = torch.where((t < case["first"]) | (t >= L - case["recent"]), math.inf, s["w"])
    key = torch.where(t < L, key, -math.inf)
    best = key.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    cut = s["lens"] > keep
    j = torch.arange(keep, device="cuda")
    if best.shape[-1] < keep:
        best = torch.nn.functional.pad(best, (0, keep - best.shape[-1]), value=n)
    src = torch.where(cut[:, None, None], best.sort(dim=-1).values, j)
    new = s["lens"].clamp(max=keep)
    live = (j < new[:, None])[:, None].expand(B, Hkv, keep)
    s["new_lens"].copy_(new)
    s["kept"].copy_(torch.where(live, src, s["kept"].long()))
    safe = src.clamp(max=n - 1)
    s["w_out"][..., :keep] = torch.where(live, s["w"].gather(-1, safe), s["w_out"][..., :keep])
    kb = s["spare"].shape[1]
    old = torch.nn.functional.pad(s["bt"], (0, max(0, kb - s["bt"].shape[1])), value=-1)[:, :kb]
    s["bt_out"].copy_(torch.where(cut[:, None], s["spare"], old))
    b, h, j = (live & cut[:, None, None]).nonzero(as_tuple=True)
    p = safe[b, h, j]
    sb, sr = s["bt"][b, p // BS].long(), p % BS
    db, dr = s["spare"][b, j // BS].long(), j % BS
    for c in ("k", "v"):
        pool = s[c + "c"]
        if case["pool"] == "fp8":                       # a page's scale is that of the rows it now holds
            x = pool.view(torch.float8_e4m3fn)[sb, h, sr].float() * s[c + "s"][sb, h][:, None]
            amax = torch.zeros_like(s[c + "s"])
            amax.view(-1).scatter_reduce_(0, db * Hkv + h, x.abs().amax(-1), "amax")
            sc = _page_scale(amax)
            s[c + "s"][db, h] = sc[db, h]
            pool[db, h, dr] = (x / sc[db, h][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            pool[db, h, dr] = pool[sb, h, sr]


def _plain_verify(case, s):
    B, n, V = case["B"], case["n"], case["V"]
    b, i = torch.arange(B, device="cuda"), torch.arange(n, device="cuda")
    x = s["x"].long()
    # comparisons and long sums in 64 bits: the token next to a border is decided by them
    px = s["p"][:, :n].gather(-1, x[..., None])[..., 0].double()
    qx = torch.ones_like(px) if s["q"] is None else s["q"].gather(-1, x[..., None])[..., 0].double()
    ok = (s["u"][:, :n].double() * qx < px) & (i < s["drafts"][:, None])
    acc = ok.long().cumprod(1).sum(1)
    p = s["p"][b, acc].double()
    at = acc.clamp(max=n - 1)
    if s["q"] is None:
        q = torch.zeros_like(p)
        q[b, x[b, at]] = 1
    else:
        q = s["q"][b, at].double()
    w = torch.where((acc < s["drafts"])[:, None], (p - q).clamp(min=0), p)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p)
    cdf = w.cumsum(-1)
    tok = (cdf <= s["u"][:, n:].double() * cdf[:, -1:]).sum(-1)
    s["acc"].copy_(acc)
    j = torch.arange(n + 1, device="cuda")
    xs = torch.nn.functional.pad(x, (0, 1), value=-1)
    s["out"].copy_(torch.where(j < acc[:, None], xs, torch.where(j == acc[:, None], tok[:, None], -1)))


# ----------------------------------------------------------------- costs
def work(case):
    op, D = case["op"], case.get("D", 0)
    es = 1 if case.get("pool") == "fp8" else 2
    if op == "rope":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        read = T * (Hq + 2 * Hkv) * D * 2 + T * (8 + 4 * case["axes"])
        written = T * Hq * D * 2 + T * 2 * Hkv * (D * es + (4 if es == 1 else 0))
        return {"bytes": read + written, "flops": T * (Hq + Hkv) * case["rotary"] * 3}
    if op == "weights":
        tokens = case["B"] * ((case["lo"] + case["hi"]) / 2 if case["lens"] == "uniform" else 1024 * math.exp(0.5) * 0.92)
        q = case["B"] * case["n_q"] * case["Hq"] * D * 2
        old = 4 if case["decay"] else 0
        return {"bytes": tokens * case["Hkv"] * (D * es + (0.25 if es == 1 else 0) + 4 + old) + q,
                "flops": tokens * case["Hq"] * case["n_q"] * (2 * D + 4)}
    if op == "evict":
        tokens = case["B"] * (case["lo"] + case["hi"]) / 2
        kept = case["B"] * min(case["keep"], (case["lo"] + case["hi"]) / 2)
        return {"bytes": case["Hkv"] * (4 * tokens + kept * (8 + 4 * (D * es))), "flops": tokens * case["Hkv"]}
    es = 4 if case["dtype"] == "f32" else 2
    rows = 2 if case["draft"] == "probs" else 1
    return {"bytes": case["B"] * case["V"] * es * rows, "flops": 3 * case["B"] * case["V"]}


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    return {"rope": _exact_rope, "weights": _exact_weights, "evict": _exact_evict,
            "verify": _exact_verify}[case["op"]](case, _inputs(case, seed))


def _exact_codes(x):
    """x [..., 16 or fewer rows, D] in 64 bits: the page's scale (fp32, as it is stored) and its E4M3 values."""
    sc = (x.abs().amax((-2, -1)) / 448).float().double()
    sc = torch.where(sc > 0, sc, torch.ones_like(sc))
    # the stored quotient is rounded to fp32 before it is encoded
    return sc, (x / sc[..., None, None]).float().to(torch.float8_e4m3fn).double()


def _exact_rope(case, s):
    half = case["rotary"] // 2
    pos, f = s["pos"].double(), torch.from_numpy(s["inv_freq"]).cuda()
    out = {}
    turned = {}
    for name in "qk":
        y = s[name].double().clone()
        for i in range(half):
            a = pos[int(s["axis"][i])] * f[i]
            lo, hi = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + half)
            x0, x1 = s[name][:, :, lo].double(), s[name][:, :, hi].double()
            z = torch.polar(torch.ones_like(a), a)[:, None] * torch.complex(x0, x1)
            y[:, :, lo], y[:, :, hi] = z.real, z.imag
        turned[name] = y
    out["q"] = turned["q"]
    blk, row = s["slots"] // BS, s["slots"] % BS
    for n, x in (("k", turned["k"]), ("v", s["v"].double())):
        pool = torch.zeros(s[n + "c"].shape, dtype=torch.float64, device="cuda")
        if case["pool"] == "fp8":
            # encoded from the row in the activations' type
            sc, val = _exact_codes(x.to(s["q"].dtype).double()[:, :, None])
            scale = s[n + "s"].double().clone()
            scale[blk] = sc
            pool[blk, :, row] = val[:, :, 0]
            out[n + "s"] = scale
        else:
            pool[blk, :, row] = x
        out[n + "c"] = pool
    return {k: out[k] for k in (("q", "kc", "vc", "ks", "vs") if case["pool"] == "fp8" else ("q", "kc", "vc"))}


def _exact_weights(case, s):
    Hkv, D, n_q = case["Hkv"], case["D"], case["n_q"]
    G = case["Hq"] // Hkv
    w = s["w"].double().clone()
    q = s["q"].double().view(case["B"], n_q, Hkv, G, D)
    for b in range(case["B"]):
        L = int(s["lens"][b])
        blocks = s["bt"][b, :(L + BS - 1) // BS].long()
        for h in range(Hkv):
            k = s["kc"][blocks, h]
            k = k.view(torch.float8_e4m3fn).double() * s["ks"][blocks, h].double()[:, None, None] \
                if case["pool"] == "fp8" else k.double()
            k = k.reshape(-1, D)[:L]
            got = torch.zeros(L, dtype=torch.float64, device="cuda")
            for i in range(n_q):
                n = L - n_q + 1 + i
                if n > 0:
                    got[:n] += torch.softmax(k[:n] @ q[b, i, h].T * s["scale"], 0).sum(1)
            old = w[b, h, :L] * case["decay"]
            old[max(0, L - n_q):] = 0
            w[b, h, :L] = old + got
    return {"w": w}


def _exact_evict(case, s):
    B, Hkv, keep, nb = case["B"], case["Hkv"], case["keep"], s["nb"]
    fp8 = case["pool"] == "fp8"
    W, lens, bt = s["w"].cpu().numpy().astype(np.float64), s["lens"].cpu().numpy(), s["bt"].cpu().numpy()
    spare = s["spare"].cpu().numpy()
    out = {n: torch.zeros(s[n][nb:].shape, dtype=torch.float64, device="cuda") for n in ("kc", "vc")}
    if fp8:
        out |= {n: torch.ones(s[n][nb:].shape, dtype=torch.float64, device="cuda") for n in ("ks", "vs")}
    w_out = s["w_out"].double().clone()
    kept = s["kept"].clone()
    tables = s["bt_out"].clone()
    for b in range(B):
        L = int(lens[b])
        row = spare[b] if L > keep else np.concatenate([bt[b], np.full(spare.shape[1], -1)])[:spare.shape[1]]
        tables[b] = torch.from_numpy(np.asarray(row, dtype=np.int32)).cuda()
        for h in range(Hkv):
            mid = range(case["first"], L - case["recent"])
            src = list(range(L))
            if L > keep:
                heavy = sorted(mid, key=lambda t: (-W[b, h, t], t))[:keep - case["first"] - case["recent"]]
                src = sorted(list(range(case["first"])) + heavy + list(range(L - case["recent"], L)))
            at = torch.tensor(src, device="cuda")
            kept[b, h, :len(src)] = at.to(torch.int32)
            w_out[b, h, :len(src)] = s["w"][b, h, at].double()
            if L <= keep:
                continue
            blk = s["bt"][b, at // BS].long()
            dst = (s["spare"][b].long() - nb)
            for c in "kv":
                x = s[c + "c"][blk, h, at % BS]
                x = x.view(torch.float8_e4m3fn).double() if fp8 else x.double()
                pages = torch.zeros(dst.numel() * BS, case["D"], dtype=torch.float64, device="cuda")
                # a value is the fp32 product of its code and its page's scale
                pages[:keep] = (x.float() * s[c + "s"][blk, h][:, None]).double() if fp8 else x
                pages = pages.view(-1, BS, case["D"])
                if fp8:
                    out[c + "s"][dst, h], pages = _exact_codes(pages)
                out[c + "c"][dst, h] = pages
    return {**{n: out[n] for n in (("kc", "vc", "ks", "vs") if fp8 else ("kc", "vc"))}, "w": w_out, "kept": kept,
            "lens": s["lens"].clamp(max=keep), "tables": tables}


def _exact_verify(case, s):
    n = case["n"]
    out, acc = s["out"].clone(), s["acc"].clone()
    for b in range(case["B"]):
        x = s["x"][b].tolist()
        r = 0
        while r < int(s["drafts"][b]):
            q = 1.0 if s["q"] is None else float(s["q"][b, r, x[r]])
            if not float(s["u"][b, r]) * q < float(s["p"][b, r, x[r]]):
                break
            r += 1
        w = s["p"][b, r].double()
        if r < int(s["drafts"][b]):
            q = torch.zeros_like(w) if s["q"] is None else s["q"][b, r].double()
            if s["q"] is None:
                q[x[r]] = 1
            left = (w - q).clamp(min=0)
            w = left if float(left.sum()) > 0 else w
        cdf = np.cumsum(w.cpu().numpy())
        out[b, :r] = s["x"][b, :r]
        out[b, r] = int(np.searchsorted(cdf, float(s["u"][b, n]) * cdf[-1], side="right"))
        acc[b] = r
    return {"tokens": out, "accepted": acc}
