"""GPU test of the cache operators used together, as a decode loop uses them:
prompts appended with rotary positions, decode steps that append, attend and
add up the tokens' weights, an eviction in place and one to new pages, more
steps with positions past the thinned cache's rows, and ART walks over the
caches in between.  A 64-bit cache kept in step on the CPU is the reference;
eviction decisions are checked against the weights the GPU holds."""
import numpy as np
import pytest
import torch

from tests import cache_ref as ref
from tests.test_gpu_split import verify

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, PAGE, WIDTH = 3, 8, 2, 128, 64, 6


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_a_decode_loop(cuda_lib, layout):
    art, dev = cuda_lib, "cuda"
    g = torch.Generator().manual_seed(11)
    pages = 2 * B * WIDTH
    perm = torch.randperm(pages, generator=g).int()
    table, spare = perm[:B * WIDTH].view(B, WIDTH).clone(), perm[B * WIDTH:].view(B, WIDTH).clone()
    kc = torch.full((pages, HKV, PAGE, D), float("nan"), dtype=torch.bfloat16, device=dev)
    vc = kc.clone()
    mass = torch.full((B, HKV, WIDTH * PAGE), 5.0, device=dev)          # appends have to clear it
    rope = art.art_rope_init(D, rot_dim=64, layout=layout, base=500000.0, scaling="by_parts", factor=8.0, original_len=8192,
                             high_turns=4.0)
    f = 500000.0 ** (-2.0 * np.arange(32) / 64)
    keep = np.clip((8192 * f / (2 * np.pi) - 1) / 3, 0, 1)
    f = keep * f + (1 - keep) * f / 8
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lens, pos = [0] * B, [0] * B
    draw = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)   # noqa: E731

    def append(new):
        seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(new)])
        slots = torch.cat([torch.arange(lens[b], lens[b] + n, dtype=torch.int32) for b, n in enumerate(new)])
        at = torch.cat([torch.arange(pos[b], pos[b] + n, dtype=torch.int32) for b, n in enumerate(new)])
        T = len(seq)
        q, k, v = 2 * draw(T, HQ, D), draw(T, HKV, D), draw(T, HKV, D)
        got = art.art_rope_append(rope, q.to(dev), k.to(dev), v.to(dev), kc, vc, table.to(dev), slots.to(dev),
                                  positions=at.to(dev), token_seq=seq.to(dev), mass=mass, device_status=status)
        torch.cuda.synchronize()
        cos, sin = ref.turn_by(f, at.numpy())
        for x, y in ((q, got), (k, kc[table[seq.long(), slots.long() // PAGE].long().to(dev), :, (slots.long() % PAGE).to(dev)])):
            want = ref.rotate(x, cos, sin, 64, layout)
            assert bool(((y.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -21 * 2 * x.abs().max()).all())
        for b, n in enumerate(new):
            lens[b] += n
            pos[b] += n
        return got

    def attend(q):
        sl = torch.tensor(lens, dtype=torch.int32, device=dev)
        before = mass.clone()
        o, e = art.art_decode_attention_split(q, kc, vc, table.to(dev), sl, mass=mass, device_status=status)
        walk, stop = art.art_decode_attention(q, kc, vc, table.to(dev), None, sl, 0.0, 0.0, 1, 1)
        torch.cuda.synchronize()
        verify(q.cpu(), kc.cpu(), vc.cpu(), table, lens, o, e, before.cpu(), mass)
        assert float((walk - o).abs().max()) < 2e-3
        return o

    append([150, 200, 64])
    for b, n in enumerate(lens):
        assert not mass[b, :, :n].any() and bool((mass[b, :, n:] == 5.0).all())
    for step in range(3):
        attend(append([1, 1, 1]))

    def evict(budget, sink, recent, moved):
        sl = torch.tensor(lens, dtype=torch.int32, device=dev)
        old_k, old_v, old_m = kc.cpu(), vc.cpu(), mass.cpu()
        kw = dict(new_page_table=spare.to(dev), new_mass=torch.empty_like(mass)) if moved else {}
        nl, kept = art.art_cache_evict(kc, vc, table.to(dev), sl, mass, budget, sink=sink, recent=recent, device_status=status,
                                       **kw)
        torch.cuda.synchronize()
        where = spare if moved else table
        new_m = kw["new_mass"] if moved else mass
        for b in range(B):
            for h in range(HKV):
                want = ref.evict_kept(old_m[b, h].tolist(), lens[b], budget, sink, recent)
                assert kept[b, h, :len(want)].tolist() == want
                n = len(want)
                for new, old in ((kc, old_k), (vc, old_v)):
                    assert torch.equal(ref.rows(new.cpu(), where, b, h, n), ref.rows(old, table, b, h, lens[b])[want])
                assert torch.equal(new_m[b, h, :n].cpu(), old_m[b, h, want]) and not new_m[b, h, n:].any()
            lens[b] = min(lens[b], budget)
        assert nl.tolist() == lens
        return where.clone(), new_m

    table, mass = evict(96, 4, 16, False)
    for step in range(2):
        attend(append([1, 1, 1]))
    table, mass = evict(70, 2, 30, True)
    attend(append([1, 3, 1])[[0, 3, 4]].contiguous())
    # the thinned cache under an importance-first ART walk
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    summ = art.art_page_summary(kc, table.to(dev), sl)
    q = draw(B, HQ, D).to(dev)
    order, _ = art.art_build_order_importance(q, summ, table.to(dev), sl, PAGE)
    out, stop = art.art_decode_attention(q, kc, vc, table.to(dev), order, sl, 0.0, 0.0, 1, 1)
    o, e = art.art_decode_attention_split(q, kc, vc, table.to(dev), sl)
    torch.cuda.synchronize()
    verify(q.cpu(), kc.cpu(), vc.cpu(), table, lens, o, e)
    assert float((out - o).abs().max()) < 2e-3 and int(status) == 0


def test_two_streams_at_once(cuda_lib):
    """The three calls on two streams at the same time, given as a stream and as a handle, on caches of their own, give
    what each gives alone."""
    art, dev, page, d = cuda_lib, "cuda", 64, 128
    g = torch.Generator().manual_seed(5)
    jobs = []
    for seed, (Hq, Hkv, n) in enumerate(((8, 2, 3000), (28, 4, 700))):
        k, v, table = ref.paged([n, n // 3], page, Hkv, d, "bf16", seed, stale=0.0, width=n // page + 2)
        jobs.append(dict(q=torch.randn(2, Hq, d, generator=g).to(dev, torch.bfloat16),
                         n=torch.randn(2, 2, Hkv, d, generator=g).to(dev, torch.bfloat16), k=k.to(dev), v=v.to(dev),
                         t=table.to(dev), s=torch.tensor([n, n // 3], dtype=torch.int32, device=dev),
                         m=torch.zeros(2, Hkv, table.shape[1] * page, device=dev)))
    rope = art.art_rope_init(d)

    def work(j, k, v, m, stream):
        got = []
        for _ in range(20):
            x = art.art_rope_append(rope, j["q"], j["n"][0], j["n"][1], k, v, j["t"], j["s"], mass=m, stream=stream)
            got += [x, *art.art_decode_attention_split(x, k, v, j["t"], j["s"], mass=m, stream=stream)]
        got += art.art_cache_evict(k, v, j["t"], j["s"], m, 150, sink=1, recent=30, stream=stream)
        return got + [k, v, m]

    copies = [[[j[x].clone() for x in "kvm"] for j in jobs] for _ in range(2)]
    alone = [work(j, *c, None) for j, c in zip(jobs, copies[0])]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [work(jobs[0], *copies[1][0], sides[0]), work(jobs[1], *copies[1][1], sides[1].cuda_stream)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("width,mode", [(4, "calls"), (4, "graph"), (40, "calls"), (40, "graph"), (700, "calls")])
def test_calls_in_a_row_equal_calls_one_by_one(cuda_lib, width, mode):
    """Every kernel of these calls may take its place before the one ahead of it has ended.  A decode loop queued without
    a wait (lengths, queries and masses changed by torch kernels in between, evictions in place and back to the other
    pages), as calls or as a replayed graph, gives the bits of the same loop with a wait after every call."""
    art, dev, steps = cuda_lib, "cuda", 12
    g = torch.Generator().manual_seed(width)
    page, Hq, Hkv, d, n = 64, 8, 2, 128, 3
    start = [min(width * page - 2 * steps - 1, 150 + 61 * b * width // 4) for b in range(n)]
    perm = torch.randperm(2 * n * width, generator=g).int()
    tables = [perm[:n * width].view(n, width).to(dev), perm[n * width:].view(n, width).to(dev)]
    k0, v0 = (torch.randn(2 * n * width, Hkv, page, d, generator=g).to(dev, torch.bfloat16) for _ in range(2))
    new = [[torch.randn(n, h, d, generator=g).to(dev, torch.bfloat16) for h in (Hq, Hkv, Hkv)] for _ in range(steps)]
    rope = art.art_rope_init(d)
    lens0 = torch.tensor(start, dtype=torch.int32, device=dev)
    kc, vc = k0.clone(), v0.clone()
    masses = [torch.zeros(n, Hkv, width * page, device=dev) for _ in range(2)]
    lens = lens0.clone()
    nl = torch.empty_like(lens)

    def reset():
        kc.copy_(k0)
        vc.copy_(v0)
        lens.copy_(lens0)
        for m in masses:
            m.zero_()

    def loop(wait):
        got, at = [], 0
        for i, (q, k, v) in enumerate(new):
            x = art.art_rope_append(rope, q, k, v, kc, vc, tables[at], lens, mass=masses[at])
            wait()
            lens.add_(1)
            x.mul_(1.5)
            wait()
            o, e = art.art_decode_attention_split(x, kc, vc, tables[at], lens, mass=masses[at])
            wait()
            got += [o, e, x]
            if i % 4 == 3:
                budget = start[0] - 7 * i
                if i % 8 == 3:
                    art.art_cache_evict(kc, vc, tables[at], lens, masses[at], budget, sink=2, recent=9, new_seq_lens=nl)
                else:
                    art.art_cache_evict(kc, vc, tables[at], lens, masses[at], budget, sink=2, recent=9, new_seq_lens=nl,
                                        new_page_table=tables[1 - at], new_mass=masses[1 - at])
                    at = 1 - at
                wait()
                lens.copy_(nl)
        return got

    reset()
    want = loop(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = [x.clone() for x in want] + [kc.clone(), vc.clone(), lens.clone()] + [m.clone() for m in masses]
    if mode == "graph":
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            reset()
            got = loop(lambda: None)
    for _ in range(4):
        if mode == "graph":
            graph.replay()
        else:
            reset()
            got = loop(lambda: None)
        torch.cuda.synchronize()
        for x, y in zip(want, got + [kc, vc, lens] + masses):
            assert torch.equal(x, y)


def test_empty_tensors_are_refused(cuda_lib):
    """A tensor of no elements is not an argument left out: no eviction in place instead of to new pages, no rotation by
    the slots, no attention without weights.  Nothing is written."""
    art, dev, SHAPE = cuda_lib, "cuda", -2
    k, v, table = ref.paged([40, 40], 16, 2, 64, "bf16", 1, stale=0.0)
    kc, vc, tg = k.to(dev), v.to(dev), table.to(dev)
    lens = torch.tensor([40, 40], dtype=torch.int32, device=dev)
    mass = torch.rand(2, 2, 48, device=dev)
    m0 = mass.clone()
    none = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=dev)      # noqa: E731
    q, n = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=dev), torch.ones(2, 2, 64, dtype=torch.bfloat16, device=dev)
    evict = lambda **kw: art.art_cache_evict(kc, vc, tg, lens, mass, 16, **kw)                            # noqa: E731
    append = lambda **kw: art.art_rope_append(art.art_rope_init(64), q, n, n, kc, vc, tg, lens, **kw)     # noqa: E731
    attend = lambda **kw: art.art_decode_attention_split(q, kc, vc, tg, lens, **kw)                       # noqa: E731
    for call, kw in ((evict, dict(new_page_table=none(2, 0, t=torch.int32))), (evict, dict(new_mass=none(2, 2, 0))),
                     (append, dict(positions=none(0, t=torch.int32))), (append, dict(token_seq=none(0, t=torch.int32))),
                     (append, dict(mass=none(2, 2, 0))), (attend, dict(mass=none(2, 2, 0))), (attend, dict(lse=none(2, 0)))):
        with pytest.raises(art.ArtError) as e:
            call(**kw)
        assert e.value.status == SHAPE, kw
    torch.cuda.synchronize()
    assert torch.equal(kc.cpu(), k) and torch.equal(vc.cpu(), v) and torch.equal(mass, m0)
