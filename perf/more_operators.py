"""Cases of the calls that a serving loop makes for whole requests over the paged cache.

Three groups: the attention of prompts over the paged cache (prefill), the pages of the pool by reference counts
(admit: free and allocate; fork: free and fork; compact), and the adjustment of logits by penalties, biases and
grammar masks with the softmax that draft verification draws from (logits).  ``run`` computes their plain forms from
elementary torch operations, or, where ``own`` is true, calls the library, bound once as a serving loop binds its
calls (``ops.prepare``).
"""
import math
import random

import numpy as np
import torch

own = False

BS = 16
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the first chunks of four short requests (the tiny batch's heads): launch latency
        dict(name="prefill_tiny", op="prefill", B=4, Hq=8, Hkv=2, D=64, dtype="f16", pool="16", lo=1, hi=256, new_lo=1,
             new_hi=48, window=0),
        # a mixed batch: chunks of prompts and single tokens of running requests, 28/4 heads
        dict(name="prefill_mixed_32", op="prefill", B=32, Hq=28, Hkv=4, D=128, dtype="f16", pool="16", lo=64, hi=8192,
             new_lo=1, new_hi=512, window=0),
        # one long prompt, all of it at once
        dict(name="prefill_prompt_16k", op="prefill", B=1, Hq=28, Hkv=4, D=128, dtype="bf16", pool="16", lo=16384,
             hi=16384, new_lo=16384, new_hi=16384, window=0),
        # the next chunks of two long prompts over a cache in E4M3
        dict(name="prefill_long_e4m3", op="prefill", B=2, Hq=28, Hkv=4, D=128, dtype="bf16", pool="fp8", lo=100000,
             hi=131072, new_lo=384, new_hi=512, window=0),
        # four requests end and four begin, in a pool of 64 pages
        dict(name="admit_tiny", op="admit", rows=4, turn=4, lo=1, hi=256, spare=0.0, grow=0),
        # a quarter of 256 long requests ends, as many begin, the others grow
        dict(name="admit_256_long", op="admit", rows=256, turn=64, lo=4096, hi=32768, spare=0.1, grow=192),
        # one step of a beam of four
        dict(name="fork_beam_4", op="fork", rows=8, pairs=3, Hkv=2, D=64, pool="16", lo=17, hi=256),
        # 32 prompts, four samples of each: the pages shared, the last one copied
        dict(name="fork_samples_96", op="fork", rows=128, pairs=96, Hkv=4, D=128, pool="16", lo=100, hi=2000),
        # a pool of 16384 pages that is half empty
        dict(name="compact_16k_pages", op="compact", rows=48, NB=16384, live=0.5, Hkv=2, D=128, pool="16"),
        # an E4M3 pool of 48k pages, four of five in use, an odd count
        dict(name="compact_48k_pages_e4m3", op="compact", rows=200, NB=49001, live=0.8, Hkv=4, D=128, pool="fp8"),
        # one request, one token: latency
        dict(name="logits_one", op="logits", B=1, n=0, V=32000, dtype="f32", probs=False, history=300, bias=8,
             mask="none"),
        # 128 requests with three drafts each: the target's distributions for draft verification
        dict(name="logits_batch_128", op="logits", B=128, n=3, V=128000, dtype="bf16", probs=True, history=4096, bias=64,
             mask="grammar"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "admit", "fork", "compact", "logits", "logits"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    pool = rng.choice(["16", "fp8"])
    if op == "prefill":
        G = rng.choice([1, 2, 3, 4, 7, 8])
        hi = _log(rng, 8, 60000)
        new_hi = min(hi, _log(rng, 1, 3000))
        # pairs of query and key, and tokens in all
        B = max(1, min(_log(rng, 1, 64), int(2e10 / (hi * new_hi * Hkv * G * D / 128)), 400000 // (hi * Hkv)))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["f16", "bf16"]), pool=pool,
                    lo=rng.randint(1, hi), hi=hi, new_lo=rng.randint(0, new_hi), new_hi=new_hi,
                    window=rng.choice([0, 0, 0, _log(rng, 1, hi)]))
    if op == "admit":
        rows = _log(rng, 1, 500)
        hi = _log(rng, 2, min(32768, 4_000_000 // rows))
        turn = rng.randint(0, rows)
        return dict(op=op, rows=rows, turn=turn, lo=rng.randint(1, hi), hi=hi, spare=rng.choice([0.0, 0.3]),
                    grow=rng.randint(0, rows - turn))
    if op == "fork":
        rows = rng.randint(2, 150)
        hi = _log(rng, 2, min(4000, 100000 // rows))
        return dict(op=op, rows=rows, pairs=rng.randint(1, rows - 1), Hkv=Hkv, D=D, pool=pool,
                    lo=rng.randint(1, hi), hi=hi)
    if op == "compact":
        NB = _log(rng, 20, 40000 // Hkv)
        return dict(op=op, rows=rng.randint(1, max(1, min(200, NB // 8))), NB=NB, live=round(rng.uniform(0.05, 0.98), 3),
                    Hkv=Hkv, D=D, pool=pool)
    V = _log(rng, 500, 130000)
    n = rng.choice([0, 0, 1, 3, 7])
    B = max(1, min(_log(rng, 1, 128), 50_000_000 // (V * (n + 1))))
    return dict(op=op, B=B, n=n, V=V, dtype=rng.choice(["f32", "bf16", "f16"]), probs=rng.random() < 0.6,
                history=_log(rng, 1, 20000), bias=rng.choice([0, 1, 17, 300]), mask=rng.choice(["none", "grammar"]))


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


def _ints(g, lo, hi, n):
    """n whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _shuffled(case, g, make):
    """A number of make(rng) for each of the case's sequences or rows: the case alone says which, the seed in what
    order, so that outputs have the same shapes whatever the seed."""
    rng = random.Random(repr([case.get(k) for k in ("op", "B", "rows", "lo", "hi", "new_lo", "new_hi", "NB")]))
    made = torch.tensor([make(rng) for _ in range(case.get("B") or case["rows"])], device="cuda")
    return made[torch.randperm(made.shape[0], generator=g, device="cuda")]


def _tables(pages, width, ids):
    """Tables of pages[r] pages a row, taken from ids in order; -1 behind them."""
    used = torch.arange(width, device="cuda")[None, :] < pages[:, None]
    t = torch.full((pages.numel(), width), -1, dtype=torch.int32, device="cuda")
    t[used] = ids[:int(pages.sum())].to(torch.int32)
    return t


def _pools(g, nb, Hkv, D, pool, dtype=torch.float16):
    """K and V pools of nb pages (E4M3 ones with their scales) whose values are of order one."""
    s = {}
    for n in "kv":
        if pool != "fp8":
            s[n + "c"] = _randn(g, (nb, Hkv, BS, D), dtype)
            continue
        s[n + "c"] = torch.empty(nb, Hkv, BS, D, dtype=torch.uint8, device="cuda")
        s[n + "s"] = torch.empty(nb, Hkv, dtype=torch.float32, device="cuda")
        for i in range(0, nb, 4096):
            x = torch.randn(min(4096, nb - i), Hkv, BS, D, generator=g, device="cuda")
            # pages of one sequence differ in how large their values are
            x *= torch.rand(x.shape[0], Hkv, 1, 1, generator=g, device="cuda") + 0.5
            sc = x.abs().amax(dim=(2, 3)) / 448
            s[n + "c"][i:i + 4096] = (x / sc[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s[n + "s"][i:i + 4096] = sc
    return s


def _inputs(case, seed):
    return {"prefill": _prepare_prefill, "admit": _prepare_admit, "fork": _prepare_fork, "compact": _prepare_compact,
            "logits": _prepare_logits}[case["op"]](case, _gen(seed))


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if own:
        s["call"] = _bind(case, s)
    return s


def _prepare_prefill(case, g):
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    dt = DT[case["dtype"]]
    count = iter(range(B))

    def request(rng):
        L = rng.randint(case["lo"], case["hi"])
        n = min(L, rng.randint(case["new_lo"], case["new_hi"]))
        return L, min(n, 1) if next(count) % 4 == 0 and B >= 4 else n     # running requests: one token each

    L, n = _shuffled(case, g, request).to(torch.int32).unbind(1)
    L = L.contiguous()
    starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    starts[1:] = n.cumsum(0)
    T = max(1, int(starts[-1]))
    pages = (L + BS - 1) // BS
    nb = int(pages.sum())
    bt = _tables(pages, (case["hi"] + BS - 1) // BS, torch.randperm(nb, generator=g, device="cuda"))
    qkv = _randn(g, (T, (Hq + 2 * Hkv) * D), dt)        # one projection's output: q is a view of it
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    q *= 1.5
    return {"q": q, "starts": starts, "lens": L, "bt": bt, "scale": float(np.float32(1 / math.sqrt(D))),
            "out": torch.zeros(T, Hq, D, dtype=dt, device="cuda"), **_pools(g, nb, Hkv, D, case["pool"], dt)}


def _prepare_admit(case, g):
    """Rows of a table of which the first ``turn`` (in a shuffled order) end and begin anew with other lengths, and
    the next ``grow`` get room for up to 64 more tokens."""
    rows, hi = case["rows"], case["hi"]
    pages = (_ints(g, case["lo"], hi, rows) + BS - 1) // BS
    width = (hi + 64 + BS - 1) // BS
    need = rows * ((hi + BS - 1) // BS) + case["grow"] * 4
    nb = max(64, int(need * (1 + case["spare"])))
    ids = torch.randperm(nb, generator=g, device="cuda")
    bt = _tables(pages, width, ids)
    ref = torch.zeros(nb, dtype=torch.int32, device="cuda")
    ref[ids[:int(pages.sum())]] = 1
    order = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
    ends, grow = order[:case["turn"]], order[case["turn"]:case["turn"] + case["grow"]]
    new = torch.cat([_ints(g, case["lo"], hi, ends.numel()), pages[grow.long()] * BS + _ints(g, 0, 64, grow.numel())])
    return {"bt": bt, "pages": pages, "ref": ref, "ends": ends.contiguous(), "rows": torch.cat([ends, grow]),
            "new": new.to(torch.int32).clamp(max=width * BS),
            "granted": torch.zeros(ends.numel() + grow.numel(), dtype=torch.int32, device="cuda")}


def _prepare_fork(case, g):
    """Some rows end; their places are taken by forks of the others."""
    rows, pairs = case["rows"], case["pairs"]
    L = _shuffled(case, g, lambda rng: rng.randint(case["lo"], case["hi"])).to(torch.int32)
    pages = (L + BS - 1) // BS
    nb = int(pages.sum()) + rows + 3
    ids = torch.randperm(nb, generator=g, device="cuda")
    bt = _tables(pages, (case["hi"] + BS - 1) // BS, ids)
    ref = torch.zeros(nb, dtype=torch.int32, device="cuda")
    ref[ids[:int(pages.sum())]] = 1
    order = torch.randperm(rows, generator=g, device="cuda").to(torch.int32)
    dst, keep = order[:pairs].contiguous(), order[pairs:]
    src = keep[torch.randint(0, rows - pairs, (pairs,), generator=g, device="cuda")].contiguous()
    return {"bt": bt, "pages": pages, "ref": ref, "lens": L, "src": src, "dst": dst,
            "granted": torch.zeros(pairs, dtype=torch.int32, device="cuda"),
            **_pools(g, nb, case["Hkv"], case["D"], case["pool"])}


def _prepare_compact(case, g):
    """Rows that share their first pages here and there, in a pool with holes."""
    rows, nb = case["rows"], case["NB"]
    live = max(1, int(nb * case["live"]))
    cut = _shuffled(case, g, lambda rng: rng.random() + 0.2)
    pages = (cut / cut.sum() * live).floor().to(torch.int32)
    width = max(1, int(pages.max()))
    bt = _tables(pages, width, torch.randperm(nb, generator=g, device="cuda"))
    shared = (pages[1::2] // 4)[:, None]                # each odd row shares a quarter with the one before it
    first = torch.arange(width, device="cuda")[None, :] < torch.minimum(shared, pages[0::2][:shared.shape[0], None])
    bt[1::2] = torch.where(first, bt[0::2][:first.shape[0]], bt[1::2])
    ref = torch.zeros(nb, dtype=torch.int32, device="cuda")
    ref.scatter_add_(0, bt[bt >= 0].long(), torch.ones_like(bt[bt >= 0]))
    return {"bt": bt, "pages": pages, "ref": ref, "bt_out": torch.full_like(bt, -1), "ref_out": torch.zeros_like(ref),
            "moved": torch.full_like(ref, -1), "live": torch.zeros(1, dtype=torch.int32, device="cuda"),
            **_pools(g, nb, case["Hkv"], case["D"], case["pool"])}


def _prepare_logits(case, g):
    B, n, V, H = case["B"], case["n"], case["V"], case["history"]
    s = {"x": (torch.randn(B, n + 1, V, generator=g, device="cuda") * 3).to(DT[case["dtype"]])}
    # text repeats itself: low token numbers far more often
    u = torch.rand(B, H + n, generator=g, device="cuda", dtype=torch.float64)
    tok = (V ** u - 1).long().clamp(max=V - 1).to(torch.int32)
    s["hist"], s["drafts"] = tok[:, :H].contiguous(), tok[:, H:].contiguous()
    s["hist_lens"] = _ints(g, H // 2, H, B)
    s["prompt_lens"] = (s["hist_lens"] * torch.rand(B, generator=g, device="cuda")).to(torch.int32)
    r = torch.rand(4, B, generator=g, device="cuda")
    s["rep"], s["pres"], s["freq"] = 1 + 0.3 * r[0], 0.8 * r[1] - 0.2, 0.5 * r[2]
    s["temp"] = torch.where(r[3] < 0.1, torch.zeros_like(r[3]), 0.3 + r[3])     # one in ten is greedy
    s["bias_t"] = torch.randint(-1, V, (B, case["bias"]), generator=g, device="cuda", dtype=torch.int32)
    s["bias_v"] = torch.randn(B, case["bias"], generator=g, device="cuda") * 4
    s["allowed"] = None
    if case["mask"] == "grammar":                       # some rows free, some down to a few tokens, some to none
        words = (V + 31) // 32
        bits = torch.randint(-2 ** 31, 2 ** 31, (B, n + 1, words), generator=g, device="cuda")
        few = torch.randint(-2 ** 31, 2 ** 31, (B, n + 1, words), generator=g, device="cuda") & 0x11
        rare = torch.rand(B, n + 1, words, generator=g, device="cuda") < 0.01
        kind = torch.randint(0, 16, (B, n + 1, 1), generator=g, device="cuda")
        bits = torch.where(kind < 8, torch.full_like(bits, -1), torch.where(kind < 12, bits, torch.where(
            rare & (kind < 15), few, torch.zeros_like(bits))))
        s["allowed"] = bits.to(torch.int32)
    s["out"] = torch.zeros(B, n + 1, V, dtype=torch.float32 if case["probs"] else DT[case["dtype"]], device="cuda")
    return s


# ---------------------------------------------------- the library's calls
def _bind_prefill(case, s):
    from paged_kv_cache_179_gb300 import ops
    s["ws"] = ops.alloc_prefill_workspace(case["B"], s["q"].shape[0], case["Hq"], case["Hkv"], case["D"], s["q"].device)
    args = (s["bt"], s["lens"], case["hi"], s["starts"], s["scale"], s["ws"])
    if case["pool"] == "fp8":
        return ops.prepare(lambda: ops.pa_prefill_fp8(s["out"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], *args,
                                                      window=case["window"]))
    return ops.prepare(lambda: ops.pa_prefill(s["out"], s["q"], s["kc"], s["vc"], *args, window=case["window"]))


def _bind_admit(case, s):
    from paged_kv_cache_179_gb300 import ops

    def body():
        ops.pa_free_pages(s["bt"], s["pages"], s["ends"], s["ref"])
        ops.pa_alloc_pages(s["bt"], s["pages"], s["rows"], s["new"], s["ref"], s["granted"])
    return ops.prepare(body)


def _bind_fork(case, s):
    from paged_kv_cache_179_gb300 import ops

    def body():
        ops.pa_free_pages(s["bt"], s["pages"], s["dst"], s["ref"])
        ops.pa_fork_pages(s["kc"], s["vc"], s["bt"], s["pages"], s["lens"], s["src"], s["dst"], s["ref"], s["granted"],
                          k_scale=s.get("ks"), v_scale=s.get("vs"))
    return ops.prepare(body)


def _bind_compact(case, s):
    from paged_kv_cache_179_gb300 import ops
    s["ws"] = ops.alloc_compact_workspace(case["NB"], s["bt"].device)
    return ops.prepare(lambda: ops.pa_compact_pages(
        s["kc"], s["vc"], s["bt"], s["pages"], s["ref"], s["bt_out"], s["ref_out"], s["moved"], s["live"], s["ws"],
        k_scale=s.get("ks"), v_scale=s.get("vs")))


def _bind_logits(case, s):
    from paged_kv_cache_179_gb300 import ops
    spec = ops.LogitsSpec(history=s["hist"], history_lens=s["hist_lens"], prompt_lens=s["prompt_lens"],
                          repetition=s["rep"], presence=s["pres"], frequency=s["freq"], temperature=s["temp"],
                          bias_tokens=s["bias_t"], bias_values=s["bias_v"], allowed=s["allowed"],
                          draft_tokens=s["drafts"])
    return ops.prepare(lambda: ops.pa_process_logits(s["out"], s["x"], spec, probs=case["probs"]))


def _bind(case, s):
    return {"prefill": _bind_prefill, "admit": _bind_admit, "fork": _bind_fork, "compact": _bind_compact,
            "logits": _bind_logits}[case["op"]](case, s)


# ------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        s["call"]()
    else:
        {"prefill": _plain_prefill, "admit": _plain_admit, "fork": _plain_fork, "compact": _plain_compact,
         "logits": _plain_logits}[case["op"]](case, s)
    return _outputs(case, s)


def _pool_outputs(case, s):
    """E4M3 codes as the values they stand for, in units of their page's scale."""
    if case["pool"] == "fp8":
        return {"kc": s["kc"].view(torch.float8_e4m3fn), "vc": s["vc"].view(torch.float8_e4m3fn), "ks": s["ks"],
                "vs": s["vs"]}
    return {"kc": s["kc"], "vc": s["vc"]}


def _outputs(case, s):
    op = case["op"]
    if op in ("prefill", "logits"):
        return {"out": s["out"]}
    if op == "admit":
        return {n: s[n] for n in ("bt", "pages", "ref", "granted")}
    if op == "fork":
        return {**{n: s[n] for n in ("bt", "pages", "ref", "lens", "granted")}, **_pool_outputs(case, s)}
    return {**{n: s[n] for n in ("bt_out", "ref_out", "moved", "live")}, **_pool_outputs(case, s)}


def _plain_prefill(case, s):
    Hkv, D, W = case["Hkv"], case["D"], case["window"]
    G = case["Hq"] // Hkv
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        blocks = s["bt"][b, :(L + BS - 1) // BS].long()
        for h in range(Hkv if n else 0):
            k, v = s["kc"][blocks, h], s["vc"][blocks, h]
            if case["pool"] == "fp8":
                k = k.view(torch.float8_e4m3fn).float() * s["ks"][blocks, h][:, None, None]
                v = v.view(torch.float8_e4m3fn).float() * s["vs"][blocks, h][:, None, None]
            k, v = k.reshape(-1, D)[:L].float(), v.reshape(-1, D)[:L].float()
            step = max(1, (1 << 27) // (G * L))         # query tokens at a time
            for i in range(0, n, step):
                m = min(step, n - i)
                at = slice(starts[b] + i, starts[b] + i + m)
                q = s["q"][at, h * G:h * G + G].float().reshape(m * G, D)
                pos = (L - n + i + torch.arange(m, device="cuda")).repeat_interleave(G)[:, None]
                j = torch.arange(L, device="cuda")[None, :]
                x = q @ k.T * s["scale"]
                x = x.masked_fill((j > pos) | ((j <= pos - W) if W else j < 0), -math.inf)
                e = (x - x.amax(-1, keepdim=True)).exp()
                o = e @ v / e.sum(-1, keepdim=True)
                s["out"][at, h * G:h * G + G] = o.view(m, G, D).to(s["out"].dtype)


def _plain_free(s, rows):
    """The pages of these rows lose an owner each, and the rows are empty."""
    rows = rows.long()
    t = s["bt"][rows]
    t = t[torch.arange(t.shape[1], device="cuda")[None, :] < s["pages"][rows][:, None]].long()
    s["ref"].scatter_add_(0, t, torch.full_like(t, -1, dtype=torch.int32))
    s["bt"][rows] = torch.where(torch.arange(s["bt"].shape[1], device="cuda")[None, :] < s["pages"][rows][:, None],
                                torch.full_like(s["bt"][rows], -1), s["bt"][rows])
    s["pages"][rows] = 0


def _plain_take(s, need):
    """The first free page of each item and whether the pool holds enough for it and those before it."""
    free = (s["ref"] == 0).nonzero()[:, 0]
    end = need.long().cumsum(0)
    return free, end - need, end <= free.numel()


def _plain_admit(case, s):
    _plain_free(s, s["ends"])
    rows = s["rows"].long()
    want = (s["new"] + BS - 1) // BS
    need = (want - s["pages"][rows]).clamp(min=0)
    free, first, ok = _plain_take(s, need)
    j = torch.arange(s["bt"].shape[1], device="cuda")[None, :]
    have = s["pages"][rows][:, None]
    new = (j >= have) & (j < want[:, None]) & ok[:, None]
    if free.numel():
        ids = free[(first[:, None] + j - have).clamp(0, free.numel() - 1)].to(torch.int32)
        s["bt"][rows] = torch.where(new, ids, s["bt"][rows])
        s["ref"][ids[new].long()] = 1
    s["pages"][rows] = torch.where(ok, torch.maximum(want, s["pages"][rows]), s["pages"][rows])
    s["granted"].copy_(ok)


def _plain_fork(case, s):
    _plain_free(s, s["dst"])
    src, dst = s["src"].long(), s["dst"].long()
    L = s["lens"][src]
    full, part = L // BS, (L % BS > 0).to(torch.int32)
    free, first, ok = _plain_take(s, part)
    j = torch.arange(s["bt"].shape[1], device="cuda")[None, :]
    t = s["bt"][src]
    share = (j < full[:, None]) & ok[:, None]
    s["ref"].scatter_add_(0, t[share].long(), torch.ones_like(t[share]))
    copy = (part > 0) & ok
    new = torch.zeros_like(src) if not free.numel() else free[first.clamp(max=free.numel() - 1)]
    old = t.gather(1, full.long().clamp(max=t.shape[1] - 1)[:, None])[:, 0].long()
    for n in ("kc", "vc", "ks", "vs"):
        if n in s:
            s[n][new[copy]] = s[n][old[copy]]
    s["ref"][new[copy]] = 1
    row = torch.where(share, t, s["bt"][dst])
    s["bt"][dst] = torch.where((j == full[:, None]) & copy[:, None], new[:, None].to(torch.int32), row)
    s["pages"][dst] = torch.where(ok, full + part, s["pages"][dst])
    s["lens"][dst] = torch.where(ok, L, s["lens"][dst])
    s["granted"].copy_(ok)


def _plain_compact(case, s):
    used = s["ref"] > 0
    n = used.sum()
    i = torch.arange(used.numel(), device="cuda")
    to = torch.where(used, i, torch.full_like(i, -1))
    src, dst = (used & (i >= n)).nonzero()[:, 0], (~used & (i < n)).nonzero()[:, 0]
    to[src] = dst
    ref = s["ref"].clone()
    ref[dst] = s["ref"][src]
    ref[src] = 0
    for c in ("kc", "vc", "ks", "vs"):
        if c in s:
            s[c][dst] = s[c][src]
    s["ref_out"].copy_(ref)
    s["moved"].copy_(to)
    s["live"].copy_(n)
    inside = torch.arange(s["bt"].shape[1], device="cuda")[None, :] < s["pages"][:, None]
    s["bt_out"].copy_(torch.where(inside, to[s["bt"].clamp(min=0).long()], s["bt"].long()))


def _plain_logits(case, s):
    B, n, V = case["B"], case["n"], case["V"]
    R = n + 1
    x = s["x"].float()
    j = torch.arange(s["hist"].shape[1], device="cuda")[None, :]
    t = s["hist"].long()
    inside = j < s["hist_lens"][:, None]
    prompt = inside & (j < s["prompt_lens"][:, None])
    seen = torch.zeros(B, 1, V, device="cuda")
    seen[:, 0].scatter_add_(1, t, prompt.float())
    count = torch.zeros(B, R, V, device="cuda")
    count.scatter_add_(2, t[:, None].expand(B, R, -1), (inside & ~prompt).float()[:, None].expand(B, R, -1))
    for i in range(1, R):                               # the drafts before a row count as its output
        count[:, i].scatter_add_(1, s["drafts"][:, :i].long(), torch.ones(B, i, device="cuda"))
    rep = s["rep"][:, None, None]
    x = torch.where((seen > 0) | (count > 0), torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["freq"][:, None, None] * count - s["pres"][:, None, None] * (count > 0)
    del seen, count
    bias = torch.zeros(B, 1, V + 1, device="cuda")
    bias[:, 0].scatter_add_(1, torch.where(s["bias_t"] < 0, V, s["bias_t"]).long(), s["bias_v"])
    x = x + bias[..., :V]
    if s["allowed"] is not None:
        v = torch.arange(V, device="cuda")
        x = x.masked_fill((s["allowed"][..., v // 32] >> (v % 32).to(torch.int32)) & 1 == 0, -math.inf)
    if case["probs"]:
        top = x.amax(-1, keepdim=True)
        d = torch.where(top > -math.inf, x - top, torch.full_like(x, -math.inf))
        temp = s["temp"][:, None, None]
        e = (d / torch.where(temp > 0, temp, torch.ones_like(temp))).exp()
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
        v = torch.arange(V, device="cuda")
        best = torch.where(d == 0, v, V).amin(-1, keepdim=True)
        x = torch.where(temp > 0, p, (v == best).float())
    s["out"].copy_(x)


# ----------------------------------------------------------------- costs
def work(case):
    op, D = case["op"], case.get("D", 0)
    es = 1 if case.get("pool") == "fp8" else 2
    if op == "prefill":
        L = (case["lo"] + case["hi"]) / 2
        n = min((case["new_lo"] + case["new_hi"]) / 2, L)
        B = case["B"]
        if B >= 4:                                      # a quarter of the sequences has one token
            B, one = B - (B + 3) // 4, (B + 3) // 4
        else:
            one = 0
        seen = min(L, case["window"] or L)
        pairs = B * n * max(seen - (n / 2 if seen == L else 0), 1) + one * seen
        cached = case["B"] * min(L, seen + n)
        return {"bytes": (B * n + one) * case["Hq"] * D * 4 + cached * case["Hkv"] * 2 * (D * es + (0.25 if es == 1 else 0)),
                "flops": pairs * case["Hq"] * 4 * D}
    if op == "admit":
        pages = (case["lo"] + case["hi"]) / 2 / BS
        # the freed pages' entries and counts, and those of the pages that take their place
        moved = 2 * case["turn"] * pages + case["grow"] * 2
        return {"bytes": moved * 12 + case["rows"] * 8, "flops": moved}
    page = case.get("Hkv", 0) * 2 * (BS * D * es + (4 if es == 1 else 0))
    if op == "fork":
        pages = (case["lo"] + case["hi"]) / 2 / BS
        return {"bytes": case["pairs"] * (2 * page * 15 / 16 + pages * 28), "flops": case["pairs"] * pages}
    if op == "compact":
        live = case["NB"] * case["live"] * 0.87         # shared pages are counted once
        moves = live * (1 - live / case["NB"])
        return {"bytes": case["NB"] * 12 + moves * 2 * page + live * 8, "flops": case["NB"]}
    rows, V = case["B"] * (case["n"] + 1), case["V"]
    es = 4 if case["dtype"] == "f32" else 2
    out = 4 if case["probs"] else es
    return {"bytes": rows * V * (es + out + (0.125 if case["mask"] == "grammar" else 0)) + case["B"] * case["history"] * 3,
            "flops": rows * V * (6 if case["probs"] else 3)}


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    return {"prefill": _exact_prefill, "admit": _exact_admit, "fork": _exact_fork, "compact": _exact_compact,
            "logits": _exact_logits}[case["op"]](case, _inputs(case, seed))


def _exact_prefill(case, s):
    Hkv, D, W = case["Hkv"], case["D"], case["window"]
    G = case["Hq"] // Hkv
    out = s["out"].double()
    lens, starts = s["lens"].cpu().numpy(), s["starts"].cpu().numpy()
    for b in range(case["B"]):
        L, n = int(lens[b]), int(starts[b + 1] - starts[b])
        if n == 0:
            continue
        page = s["bt"][b][torch.arange(L, device="cuda") // BS].long()
        row = torch.arange(L, device="cuda") % BS
        for h in range(Hkv):
            kv = []
            for c in "kv":
                x = s[c + "c"][page, h, row]
                kv.append(x.view(torch.float8_e4m3fn).double() * s[c + "s"][page, h].double()[:, None]
                          if case["pool"] == "fp8" else x.double())
            for i in range(0, n, 256):                  # 256 queries at a time, the keys that they can see
                m = min(256, n - i)
                p0 = L - n + i
                lo, hi = max(0, p0 - W + 1) if W else 0, p0 + m
                q = s["q"][starts[b] + i:starts[b] + i + m, h * G:(h + 1) * G].double()
                x = torch.einsum("mgd,jd->mgj", q, kv[0][lo:hi]) * s["scale"]
                d = p0 + torch.arange(m, device="cuda")[:, None] - torch.arange(lo, hi, device="cuda")
                x.masked_fill_(~((d >= 0) & ((d < W) if W else (d >= 0)))[:, None], -math.inf)
                out[starts[b] + i:starts[b] + i + m, h * G:(h + 1) * G] = torch.einsum(
                    "mgj,jd->mgd", torch.softmax(x, -1), kv[1][lo:hi])
    return {"out": out}


def _host(s, *names):
    return [s[n].cpu().numpy().copy() for n in names]


def _back(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _exact_free(bt, pages, ref, rows):
    for r in rows:
        for j in range(pages[r]):
            ref[bt[r, j]] -= 1
            bt[r, j] = -1
        pages[r] = 0


def _exact_admit(case, s):
    bt, pages, ref, ends, rows, new, granted = _host(s, "bt", "pages", "ref", "ends", "rows", "new", "granted")
    _exact_free(bt, pages, ref, ends)
    free = [int(p) for p in np.flatnonzero(ref == 0)]
    at, full = 0, False
    for i, r in enumerate(rows):
        want = -(-int(new[i]) // BS)
        need = max(0, want - int(pages[r]))
        full = full or at + need > len(free)
        granted[i] = 0 if full else 1
        if full:
            continue
        for p in free[at:at + need]:
            bt[r, pages[r]] = p
            pages[r] += 1
            ref[p] = 1
        at += need
    return {"bt": _back(bt), "pages": _back(pages), "ref": _back(ref), "granted": _back(granted)}


def _exact_pools(case, s):
    """The pools and scales in 64 bits (E4M3 codes as values)."""
    if case["pool"] == "fp8":
        return {"kc": s["kc"].view(torch.float8_e4m3fn).double(), "vc": s["vc"].view(torch.float8_e4m3fn).double(),
                "ks": s["ks"].double(), "vs": s["vs"].double()}
    return {"kc": s["kc"].double(), "vc": s["vc"].double()}


def _exact_fork(case, s):
    bt, pages, ref, lens, src, dst, granted = _host(s, "bt", "pages", "ref", "lens", "src", "dst", "granted")
    pools = _exact_pools(case, s)
    _exact_free(bt, pages, ref, dst)
    free = [int(p) for p in np.flatnonzero(ref == 0)]
    full = False
    for i, (a, c) in enumerate(zip(src, dst)):
        L = int(lens[a])
        full = full or (L % BS > 0 and not free)
        granted[i] = 0 if full else 1
        if full:
            continue
        for j in range(L // BS):
            bt[c, j] = bt[a, j]
            ref[bt[a, j]] += 1
        if L % BS:
            p = free.pop(0)
            for pool in pools.values():
                pool[p] = pool[int(bt[a, L // BS])]
            bt[c, L // BS] = p
            ref[p] = 1
        pages[c] = -(-L // BS)
        lens[c] = L
    return {"bt": _back(bt), "pages": _back(pages), "ref": _back(ref), "lens": _back(lens), "granted": _back(granted),
            **pools}


def _exact_compact(case, s):
    bt, pages, ref = _host(s, "bt", "pages", "ref")
    pools = _exact_pools(case, s)
    live = int((ref > 0).sum())
    to = np.where(ref > 0, np.arange(ref.size), -1).astype(np.int32)
    hole = 0
    pairs = []
    for p in range(live, ref.size):
        if ref[p] > 0:
            while ref[hole] > 0:
                hole += 1
            pairs.append((p, hole))
            to[p] = hole
            hole += 1
    new = ref.copy()
    for p, h in pairs:
        new[h], new[p] = ref[p], 0
    if pairs:
        a, b = _back(np.array(pairs, dtype=np.int64)).unbind(1)
        for pool in pools.values():
            pool[b] = pool[a]
    for r in range(bt.shape[0]):
        bt[r, :pages[r]] = to[bt[r, :pages[r]]]
    return {"bt_out": _back(bt), "ref_out": _back(new), "moved": _back(to),
            "live": torch.tensor([live], dtype=torch.int32, device="cuda"), **pools}


def _exact_logits(case, s):
    out = s["out"].double()
    hist, drafts, hl, pl = _host(s, "hist", "drafts", "hist_lens", "prompt_lens")
    V = case["V"]
    for b in range(case["B"]):
        r, f, p, temp = (float(s[n][b]) for n in ("rep", "freq", "pres", "temp"))
        bias = np.zeros(V)
        for t, v in zip(s["bias_t"][b].tolist(), s["bias_v"][b].tolist()):
            if t >= 0:
                bias[t] += v
        for i in range(case["n"] + 1):
            c = np.bincount(np.concatenate([hist[b, pl[b]:hl[b]], drafts[b, :i]]), minlength=V)
            seen = (c > 0) | (np.bincount(hist[b, :pl[b]], minlength=V) > 0)
            x = s["x"][b, i].double()
            x = torch.where(_back(seen), torch.where(x > 0, x / r, x * r), x)
            x = x - f * _back(c) - p * _back(c > 0) + _back(bias)
            if s["allowed"] is not None:
                ok = np.unpackbits(s["allowed"][b, i].cpu().numpy().view(np.uint8), bitorder="little")[:V]
                x[_back(ok) == 0] = -math.inf
            if case["probs"]:
                if float(x.max()) == -math.inf:
                    x = torch.zeros_like(x)
                elif temp > 0:
                    x = torch.softmax(x / temp, -1)
                else:
                    first = int((x == x.max()).nonzero()[0])
                    x = torch.zeros_like(x)
                    x[first] = 1
            out[b, i] = x
    return {"out": out}
