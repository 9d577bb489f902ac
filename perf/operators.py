"""The cache operators' workloads: rotary positions with the append to the
paged K/V cache, exact decode attention split over the cache's length, and
eviction by accumulated attention weight.

``listed()`` names fixed cases, ``draw(rng)`` gives others of the same ranges,
``prepare(case, seed)`` makes the inputs, ``run(state)`` is one pass: the
framework's calls where ``own`` is true, else the same operator in elementary
torch operations.  ``exact(case, seed)`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one token for each of eight sequences whose caches were thinned (positions far beyond the cache rows)
        dict(name="append decode", op="append", dtype="bf16", B=8, new_min=1, new_max=1, cached=4096, far=120000, lens_seed=1,
             Hq=32, Hkv=8, d=128, rot=128, layout="half", scaling="by_parts", factor=8.0, page=64, mass=True),
        # a ragged prompt chunk of an fp32 model that rotates half of each head, neighbouring channels paired
        dict(name="append chunk f32", op="append", dtype="f32", B=3, new_min=300, new_max=1500, cached=700, far=0, lens_seed=2,
             Hq=4, Hkv=4, d=64, rot=32, layout="interleaved", scaling="none", factor=1.0, page=16, mass=False),
        # prompts of a long-context model, written in one go
        dict(name="append prompt", op="append", dtype="bf16", B=4, new_min=4096, new_max=8192, cached=0, far=0, lens_seed=3,
             Hq=28, Hkv=4, d=128, rot=128, layout="half", scaling="ntk", factor=4.0, page=64, mass=False),
        # the smallest cache this repository walks (its tiny_fp32 shape): latency
        dict(name="attend tiny", op="attend", dtype="f32", B=1, lmin=1024, lmax=1024, lens_seed=1, Hq=4, Hkv=4, d=64, page=16,
             mass=False),
        # eight sequences of 8192 tokens (llama8b_b8)
        dict(name="attend batch", op="attend", dtype="bf16", B=8, lmin=8192, lmax=8192, lens_seed=1, Hq=32, Hkv=8, d=128, page=64,
             mass=False),
        # few units, very long caches (qwen7b_b4): the split has to fill the card
        dict(name="attend long", op="attend", dtype="bf16", B=4, lmin=131072, lmax=131072, lens_seed=1, Hq=28, Hkv=4, d=128,
             page=64, mass=False),
        # a ragged serving batch (mistral7b_b128's lengths, a quarter of its sequences)
        dict(name="attend ragged", op="attend", dtype="bf16", B=32, lmin=1024, lmax=16384, lens_seed=4, Hq=32, Hkv=8, d=128,
             page=64, mass=False),
        # the step that also keeps each token's accumulated weight, odd lengths
        dict(name="attend weights", op="attend", dtype="bf16", B=8, lmin=5001, lmax=8191, lens_seed=5, Hq=32, Hkv=8, d=128, page=64,
             mass=True),
        # wide heads, few of them, with weights
        dict(name="attend weights wide", op="attend", dtype="bf16", B=2, lmin=20001, lmax=30011, lens_seed=6, Hq=16, Hkv=2, d=256,
             page=32, mass=True),
        # a small fp32 cache cut to a quarter
        dict(name="evict small f32", op="evict", dtype="f32", B=1, lmin=1024, lmax=1024, lens_seed=1, Hkv=4, d=64, page=16,
             budget=256, sink=4, recent=64),
        # prompts of a batch cut to a quarter after prefill
        dict(name="evict batch", op="evict", dtype="bf16", B=8, lmin=6000, lmax=8192, lens_seed=7, Hkv=8, d=128, page=64,
             budget=2048, sink=4, recent=256),
        # very long prompts cut to an eighth
        dict(name="evict long", op="evict", dtype="bf16", B=4, lmin=100001, lmax=131072, lens_seed=8, Hkv=4, d=128, page=64,
             budget=16384, sink=4, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    es = 2 if dtype == "bf16" else 4
    page = rng.choice([16, 16, 24, 32, 64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    seed = rng.randrange(1 << 20)
    if op == "append":
        d = rng.choice([64, 96, 128, 128, 256])
        rot = rng.choice([d, d, d // 2, d // 4, 2 * rng.randrange(1, d // 2)])
        G = rng.choice([1, 2, 3, 4, 7, 8])
        B = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
        while B * new * (2 * Hkv * G + 4 * Hkv) * d * es > 350e6:
            new = max(1, new // 2)
            B = max(1, B // 2)
        scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
        return dict(op=op, dtype=dtype, B=B, new_min=max(1, new // 2), new_max=new, cached=_log(rng, 1, 4096),
                    far=rng.choice([0, rng.randrange(1, 500000)]), lens_seed=seed, Hq=Hkv * G, Hkv=Hkv, d=d, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]), page=page, mass=rng.random() < 0.5)
    if op == "attend":
        d = rng.choice([64, 128, 128, 256])
        G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        B = _log(rng, 1, 64)
        lmax = _log(rng, 1, 131072)
        while B * lmax * Hkv * d * es * 2 > 1000e6:
            if B > 1 and rng.random() < 0.5:
                B //= 2
            else:
                lmax //= 2
        return dict(op=op, dtype=dtype, B=B, lmin=rng.choice([1, max(1, lmax // 2), lmax]), lmax=lmax, lens_seed=seed,
                    Hq=Hkv * G, Hkv=Hkv, d=d, page=page, mass=rng.random() < 0.4)
    d = rng.choice([64, 128, 128, 256])
    B = _log(rng, 1, 32)
    lmax = _log(rng, 64, 131072)
    while B * lmax * Hkv * d * es > 500e6:
        if B > 1 and rng.random() < 0.5:
            B //= 2
        else:
            lmax //= 2
    budget = max(2, int(lmax * rng.uniform(0.05, 1.1)))
    recent = rng.randrange(0, budget // 2 + 1)
    return dict(op=op, dtype=dtype, B=B, lmin=max(1, lmax // 2), lmax=lmax, lens_seed=seed, Hkv=Hkv, d=d, page=page,
                budget=budget, sink=rng.choice([0, 1, min(4, budget - recent)]), recent=recent)


# ----------------------------------------------------------------- inputs ----

def _lengths(lo, hi, B, seed):
    """B lengths in [lo, hi], the first of them hi."""
    r = random.Random(seed)
    return [hi] + [r.randint(lo, hi) for _ in range(B - 1)]


def _table(blocks, spare, gen, dev, width=None):
    """Page table [B, width] of randomly scattered pages (-1 behind each sequence) and `spare` further page numbers."""
    total = sum(blocks) + spare
    perm = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.full((len(blocks), width or max(max(blocks), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.to(dev), perm[at:], total


def _rope_frequencies(case):
    """Radians a position for each channel pair (64 bits), scaled for long contexts."""
    rot, base, factor = case["rot"], 500000.0, case["factor"]
    i = np.arange(rot // 2, dtype=np.float64)
    if case["scaling"] == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "by_parts":    # pairs that turn often keep their frequency, slow ones are stretched
        turns = 8192 * f / (2.0 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / factor
    return f


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "by_parts" else 1.0


def prepare(case, seed):
    dev = _device()
    cpu = torch.Generator().manual_seed(int(seed) * 2 + 1)
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt, page, Hkv, d, B = _DT[case["dtype"]], case["page"], case["Hkv"], case["d"], case["B"]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    def exponential(*shape):
        return -torch.log1p(-torch.rand(*shape, generator=gen, device=dev))

    if case["op"] == "append":
        r, where = random.Random(int(seed)), random.Random(case["lens_seed"] + 1)
        new = _lengths(case["new_min"], case["new_max"], B, case["lens_seed"])
        start = [where.randint(0, case["cached"]) for _ in range(B)]
        offset = [r.randint(0, case["far"]) for _ in range(B)]
        table, _, pages = _table([-(-(s + n) // page) for s, n in zip(start, new)], 0, cpu, dev,
                                 -(-(case["cached"] + case["new_max"]) // page))
        seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(new)])
        slots = torch.cat([torch.arange(s, s + n, dtype=torch.int32) for s, n in zip(start, new)])
        positions = slots + torch.cat([torch.full((n,), o, dtype=torch.int32) for o, n in zip(offset, new)])
        T = sum(new)
        st = dict(case=case, q=normal(T, case["Hq"], d), k=normal(T, Hkv, d), v=normal(T, Hkv, d),
                  k_cache=normal(pages, Hkv, page, d), v_cache=normal(pages, Hkv, page, d), table=table, seq=seq.to(dev),
                  slots=slots.to(dev), positions=positions.to(dev), mass=None,
                  freq=torch.from_numpy(_rope_frequencies(case)).to(dev), amplitude=_amplitude(case))
        if case["mass"]:
            st["mass"] = exponential(B, Hkv, table.shape[1] * page)
        if own:
            import kv_cache_early_art_b200 as art
            st["rope"] = art.art_rope_init(d, rot_dim=case["rot"], layout=case["layout"], base=500000.0,
                                           scaling=case["scaling"], factor=case["factor"], original_len=8192,
                                           low_turns=1.0, high_turns=4.0, amplitude=st["amplitude"])
        return st

    lens = _lengths(case["lmin"], case["lmax"], B, case["lens_seed"])
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    blocks = [-(-n // page) for n in lens]
    if case["op"] == "attend":
        table, _, pages = _table(blocks, 0, cpu, dev)
        st = dict(case=case, q=normal(B, case["Hq"], d) * 2, k_cache=normal(pages, Hkv, page, d),
                  v_cache=normal(pages, Hkv, page, d), table=table, seq_lens=seq_lens, mass=None)
        if case["mass"]:
            st["mass"] = 0.1 * exponential(B, Hkv, table.shape[1] * page)
        return st

    keep = [-(-min(n, case["budget"]) // page) for n in lens]
    table, rest, pages = _table(blocks, sum(keep), cpu, dev)
    fresh = torch.full((B, max(keep)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(keep):
        fresh[b, :n] = rest[at:at + n]
        at += n
    # accumulated weights: heavy tailed, many of them small and equal
    mass = exponential(B, Hkv, table.shape[1] * page).square()
    mass = torch.where(mass < 1.0, torch.round(mass * 64) / 64, mass)
    return dict(case=case, k_cache=normal(pages, Hkv, page, d), v_cache=normal(pages, Hkv, page, d), table=table,
                seq_lens=seq_lens, mass=mass, fresh=fresh.to(dev),
                new_mass=torch.zeros(B, Hkv, fresh.shape[1] * page, device=dev))


# ------------------------------------------------------------ plain forms ----

def _rotate(x, cos, sin, rot, layout):
    """x [T, H, d] rotated by [T, rot / 2] cosines and sines, in x's precision."""
    cos, sin = cos[:, None, :], sin[:, None, :]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_append(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freq"][None, :]
    cos, sin = (s["amplitude"] * torch.cos(angle)).float(), (s["amplitude"] * torch.sin(angle)).float()
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["layout"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cos, sin, c["rot"], c["layout"]).to(s["k"].dtype)
    seq, slot = s["seq"].long(), s["slots"].long()
    pg, row = s["table"][seq, slot // c["page"]].long(), slot % c["page"]
    s["k_cache"][pg, :, row] = k
    s["v_cache"][pg, :, row] = s["v"]
    got = [q, s["k_cache"], s["v_cache"]]
    if s["mass"] is not None:
        s["mass"][seq, :, slot] = 0.0
        got.append(s["mass"])
    return got


def _plain_attend(s):
    c = s["case"]
    B, Hq, d = s["q"].shape
    Hkv, G = c["Hkv"], c["Hq"] // c["Hkv"]
    pg = s["table"].clamp(min=0).long()
    k = s["k_cache"][pg].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d).float()
    x = torch.matmul(s["q"].float().view(B, Hkv, G, d), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    del k
    live = torch.arange(x.shape[-1], device=x.device)[None, :] < s["seq_lens"][:, None]
    x = x.masked_fill(~live[:, None, None, :], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(dim=-1, keepdim=True)
    v = s["v_cache"][pg].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d).float()
    v = v.masked_fill(~live[:, None, :, None], 0.0)
    w = e / total.clamp(min=torch.finfo(torch.float32).tiny)
    out = torch.matmul(w, v).reshape(B, Hq, d)
    lse = (top + torch.log(total)).reshape(B, Hq)
    if s["mass"] is None:
        return [out, lse]
    s["mass"] += w.sum(dim=2)
    return [out, lse, s["mass"]]


def _plain_evict(s):
    c = s["case"]
    B, Hkv, S = s["mass"].shape
    page, budget, dev = c["page"], c["budget"], s["mass"].device
    t = torch.arange(S, device=dev)
    L = s["seq_lens"].long()[:, None]
    safe = (t < c["sink"]) | (t >= L - c["recent"])
    key = torch.where(safe[:, None], torch.full_like(s["mass"], math.inf), s["mass"])
    key = key.masked_fill(~(t < L)[:, None], -math.inf)
    best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    n = torch.clamp(L, max=budget)                                              # [B, 1]
    live = torch.arange(best.shape[-1], device=dev) < n                         # [B, budget]
    best = torch.where(live[:, None], best, torch.full_like(best, S))
    best = torch.sort(best, dim=-1).values
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device=dev)
    kept[..., :best.shape[-1]] = torch.where(live[:, None], best, torch.full_like(best, -1)).int()
    b, h, i = torch.nonzero(kept >= 0, as_tuple=True)
    src = kept[b, h, i].long()
    sp, dp = s["table"][b, src // page].long(), s["fresh"][b, i // page].long()
    s["k_cache"][dp, h, i % page] = s["k_cache"][sp, h, src % page]
    s["v_cache"][dp, h, i % page] = s["v_cache"][sp, h, src % page]
    s["new_mass"].zero_()
    s["new_mass"][b, h, i] = s["mass"][b, h, src]
    return [s["k_cache"], s["v_cache"], s["new_mass"], n[:, 0].int(), kept]


# -------------------------------------------------------------------- run ----

def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "evict": _plain_evict}[op](s)
    import kv_cache_early_art_b200 as art
    if op == "append":
        q = art.art_rope_append(s["rope"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["slots"],
                                positions=s["positions"], token_seq=s["seq"], mass=s["mass"])
        got = [q, s["k_cache"], s["v_cache"]]
        return got if s["mass"] is None else got + [s["mass"]]
    if op == "attend":
        out, lse = art.art_decode_attention_split(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                                                  mass=s["mass"])
        return [out, lse] if s["mass"] is None else [out, lse, s["mass"]]
    c = s["case"]
    new_lens, kept = art.art_cache_evict(s["k_cache"], s["v_cache"], s["table"], s["seq_lens"], s["mass"], c["budget"],
                                         sink=c["sink"], recent=c["recent"], new_page_table=s["fresh"],
                                         new_mass=s["new_mass"])
    return [s["k_cache"], s["v_cache"], s["new_mass"], new_lens, kept]


# ------------------------------------------------------------------- work ----

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "append":
        T = sum(_lengths(case["new_min"], case["new_max"], case["B"], case["lens_seed"]))
        return {"bytes": T * ((2 * case["Hq"] + 4 * Hkv) * d * es + 16 + (4 * Hkv if case["mass"] else 0)),
                "flops": 3 * T * (case["Hq"] + Hkv) * case["rot"]}
    lens = _lengths(case["lmin"], case["lmax"], case["B"], case["lens_seed"])
    if case["op"] == "attend":
        Hq = case["Hq"]
        n = sum(lens) * Hkv * (2 * d * es + (8 if case["mass"] else 0)) + case["B"] * Hq * (d * (es + 4) + 4)
        return {"bytes": n + sum(4 * -(-x // case["page"]) + 4 for x in lens), "flops": 4 * Hq * d * sum(lens)}
    kept = sum(min(x, case["budget"]) for x in lens)
    return {"bytes": Hkv * (4 * sum(lens) + kept * (4 * d * es + 8)), "flops": 0}


# ------------------------------------------------------- 64-bit definition ----

def _rows(s, table, b, n):
    """Pages and rows of the first n tokens of sequence b."""
    t = torch.arange(n, device=table.device)
    return table[b, t // s["case"]["page"]].long(), t % s["case"]["page"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        T, rot = s["q"].shape[0], case["rot"]
        angle = np.multiply.outer(s["positions"].cpu().numpy().astype(np.float64), _rope_frequencies(case))
        turn = torch.from_numpy(_amplitude(case) * np.exp(1j * angle)).to(s["q"].device)[:, None, :]

        def turned(x):
            x = x.double().clone()
            first = slice(0, rot // 2) if case["layout"] == "half" else slice(0, rot, 2)
            second = slice(rot // 2, rot) if case["layout"] == "half" else slice(1, rot, 2)
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        q, k = turned(s["q"]), turned(s["k"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        mass = None if s["mass"] is None else s["mass"].double()
        new = _lengths(case["new_min"], case["new_max"], case["B"], case["lens_seed"])
        at = 0
        for b, n in enumerate(new):
            slot = s["slots"][at:at + n].long()
            pg, row = s["table"][b, slot // case["page"]].long(), slot % case["page"]
            kc[pg, :, row] = k[at:at + n]
            vc[pg, :, row] = s["v"][at:at + n].double()
            if mass is not None:
                mass[b, :, slot] = 0.0
            at += n
        assert at == T
        return [q, kc, vc] if mass is None else [q, kc, vc, mass]
    lens = _lengths(case["lmin"], case["lmax"], case["B"], case["lens_seed"])
    if case["op"] == "attend":
        B, Hq, d = s["q"].shape
        Hkv, G = case["Hkv"], Hq // case["Hkv"]
        out = torch.zeros(B, Hq, d, dtype=torch.float64, device=s["q"].device)
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=s["q"].device)
        mass = None if s["mass"] is None else s["mass"].double()
        for b, n in enumerate(lens):
            pg, row = _rows(s, s["table"], b, n)
            for h in range(Hkv):
                k, v = s["k_cache"][pg, h, row].double(), s["v_cache"][pg, h, row].double()
                x = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, dim=-1)
                p = torch.softmax(x, dim=-1)
                out[b, h * G:(h + 1) * G] = p @ v
                if mass is not None:
                    mass[b, h, :n] += p.sum(dim=0)
        return [out, lse] if mass is None else [out, lse, mass]
    kc, vc, nm = s["k_cache"].double(), s["v_cache"].double(), s["new_mass"].double()
    new_lens = torch.tensor([min(n, case["budget"]) for n in lens], dtype=torch.int32)
    kept = np.full((case["B"], case["Hkv"], case["budget"]), -1, dtype=np.int32)
    mass = s["mass"].cpu().numpy().astype(np.float64)
    for b, n in enumerate(lens):
        m = min(n, case["budget"])
        dp, drow = _rows(s, s["fresh"], b, m)
        for h in range(case["Hkv"]):
            t = np.arange(n)
            safe = (t < case["sink"]) | (t >= n - case["recent"])
            order = np.lexsort((t, -mass[b, h, :n], ~safe))     # protected first, then by weight, ties by index
            stay = np.sort(order[:m])
            kept[b, h, :m] = stay
            src = torch.from_numpy(stay).to(kc.device)
            sp, srow = s["table"][b, src // case["page"]].long(), src % case["page"]
            kc[dp, h, drow] = kc[sp, h, srow]
            vc[dp, h, drow] = vc[sp, h, srow]
            nm[b, h, :m] = s["mass"][b, h, src].double()
    return [kc, vc, nm, new_lens, torch.from_numpy(kept)]
