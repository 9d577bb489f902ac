"""GPU tests of art_cache_evict against its definition: kept tokens, moved
rows and masses have to be equal bit for bit (everything is copied)."""
import math

import pytest
import torch

from tests import cache_ref as ref

pytestmark = pytest.mark.gpu


def weights(B, Hkv, width, seed, kind="ties"):
    g = torch.Generator().manual_seed(seed)
    m = torch.rand(B, Hkv, width, generator=g)
    if kind == "ties":
        m = torch.where(m < 0.7, torch.round(m * 8) / 8, m)
    return m


def run(art, lens, budget, *, sink=0, recent=0, dtype="bf16", Hkv=2, d=64, page=16, seed=0, mass=None, in_place=False,
        width=None, kind="ties"):
    B = len(lens)
    k, v, table = ref.paged(lens, page, Hkv, d, dtype, seed, stale=7.0, width=width)
    S = table.shape[1] * page
    m0 = weights(B, Hkv, S, seed, kind) if mass is None else mass
    keep = [min(max(0, n), budget) for n in lens]
    want_k, want_v = k.clone(), v.clone()
    most = min(budget, S)
    if in_place:
        target = table
    else:
        blocks = [-(-n // page) for n in keep]
        add = sum(blocks) + 2
        g = torch.Generator().manual_seed(seed + 7)
        grow = lambda c: torch.cat([c, torch.full((add, *c.shape[1:]), -2.0, dtype=c.dtype)])   # noqa: E731
        k, v, want_k, want_v = (grow(c) for c in (k, v, want_k, want_v))
        fresh = torch.randperm(add, generator=g)[:sum(blocks)] + want_k.shape[0] - add
        target = torch.full((B, -(-most // page)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(blocks):
            target[b, :n] = fresh[at:at + n]
            at += n
    nm_width = S if in_place else target.shape[1] * page + 3
    want_m = torch.zeros(B, Hkv, nm_width)
    want_kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            kept = ref.evict_kept(m0[b, h].tolist(), n, budget, sink, recent)
            want_kept[b, h, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
            src, dst = torch.tensor(kept, dtype=torch.long), torch.arange(len(kept))
            want_m[b, h, :len(kept)] = m0[b, h, src]
            sp, dp = table[b, src // page].long(), target[b, dst // page].long()
            want_k[dp, h, dst % page] = k[sp, h, src % page]
            want_v[dp, h, dst % page] = v[sp, h, src % page]
    dev = "cuda"
    kc, vc, mg = k.to(dev), v.to(dev), m0.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new_mass = None if in_place else torch.full((B, Hkv, nm_width), 4.0, device=dev)
    nl, kept = art.art_cache_evict(kc, vc, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), mg, budget,
                                   sink=sink, recent=recent, new_page_table=None if in_place else target.to(dev),
                                   new_mass=new_mass, device_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert nl.cpu().tolist() == keep
    assert torch.equal(kept.cpu(), want_kept)
    assert torch.equal((mg if in_place else new_mass).cpu(), want_m)
    if not in_place:
        assert torch.equal(mg.cpu().nan_to_num(nan=-9.0), m0.nan_to_num(nan=-9.0))
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v)


PLACES = pytest.mark.parametrize("in_place", [False, True])


@PLACES
@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([100, 64, 33, 1, 0], 32, 4, 8), ([100, 64, 33, 1, 0], 1, 0, 0), ([1000, 999], 999, 0, 0), ([40], 40, 20, 20),
    ([257], 256, 0, 255), ([5, 300], 20, 20, 0), ([5, 300], 20, 0, 20), ([31, 32, 33, 65, 500], 64, 1, 3), ([-3, 90], 10, 2, 2)])
def test_lengths_budgets_and_protected_tokens(cuda_lib, in_place, lens, budget, sink, recent):
    run(cuda_lib, lens, budget, sink=sink, recent=recent, in_place=in_place, seed=budget)


@PLACES
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 8), ("bf16", 72), ("f32", 64), ("f32", 256), ("bf16", 256)])
@pytest.mark.parametrize("page", [1, 24, 64])
def test_types_rows_and_pages(cuda_lib, in_place, dtype, d, page):
    run(cuda_lib, [150, 77], 50, sink=2, recent=10, dtype=dtype, d=d, page=page, in_place=in_place, seed=d)


@PLACES
@pytest.mark.parametrize("L", [9000, 20011, 70001])
def test_clusters(cuda_lib, in_place, L):
    """Sequences spread over 2, 4 and 8 CTAs, next to short ones."""
    run(cuda_lib, [L, 3, L // 2 + 1], L // 3, sink=4, recent=100, Hkv=1, d=8, in_place=in_place, seed=L)


@PLACES
def test_table_wider_than_the_sequences(cuda_lib, in_place):
    """The cluster and its slices follow the table's width, the work the lengths."""
    run(cuda_lib, [50, 700], 40, sink=1, recent=5, in_place=in_place, width=1200)


@PLACES
@pytest.mark.parametrize("case", ["equal", "zeros", "signs", "special"])
def test_weights(cuda_lib, in_place, case):
    """All equal (the oldest stay), zeros of both signs, negative ones, NaN and infinities."""
    g = torch.Generator().manual_seed(1)
    m = torch.randn(2, 2, 208, generator=g)
    if case == "equal":
        m = torch.full_like(m, 0.25)
    if case == "zeros":
        m = torch.where(m > 0.5, torch.tensor(0.0), torch.tensor(-0.0))
    if case == "special":
        m[:, :, ::7] = math.nan
        m[:, 0, 1::9] = math.inf
        m[:, :, 2::11] = -math.inf
        m[:, 1, 3::5] = torch.finfo(torch.float32).min
    if case == "special" and in_place:
        m = m.nan_to_num(nan=-1e30)       # compared with ==
    if case == "special" and not in_place:
        m2 = m.clone()
        m2[m2 != m2] = -math.inf          # a NaN must not be among the kept here: they are the first to go
        kept_nan = any(math.isnan(m[b, h, t]) for b in range(2) for h in range(2)
                       for t in ref.evict_kept(m[b, h].tolist(), 200, 90, 0, 0))
        assert not kept_nan
    run(cuda_lib, [200, 201], 90, mass=m, in_place=in_place)


def test_nan_weights_go_first_but_may_stay(cuda_lib):
    """With room for all numbers, the oldest of the NaN tokens stay."""
    m = torch.rand(1, 1, 64)
    m[0, 0, 10:30] = math.nan
    dev = "cuda"
    k, v, table = ref.paged([64], 16, 1, 64, "bf16", 0, stale=0.0)
    mg = m.to(dev)
    _, kept = cuda_lib.art_cache_evict(k.to(dev), v.to(dev), table.to(dev), torch.tensor([64], dtype=torch.int32, device=dev),
                                       mg, 50)
    torch.cuda.synchronize()
    assert kept[0, 0].tolist() == list(range(16)) + list(range(30, 64))


def test_largest_length(cuda_lib):
    """The longest table supported: eight full slices."""
    S = 393216
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(1)
    k = torch.randn(S // 64, 1, 64, 8, generator=g, device=dev).to(torch.bfloat16)
    table = torch.arange(S // 64, dtype=torch.int32, device=dev)[None]
    mass = torch.rand(1, 1, S, generator=g, device=dev)
    m0, k0 = mass.clone(), k.clone()
    budget = 100001
    nl, kept = cuda_lib.art_cache_evict(k, k.clone(), table, torch.tensor([S], dtype=torch.int32, device=dev), mass, budget)
    torch.cuda.synchronize()
    best = torch.sort(m0[0, 0], descending=True, stable=True).indices[:budget].sort().values
    assert torch.equal(kept[0, 0].long(), best)
    assert torch.equal(mass[0, 0, :budget], m0[0, 0, best]) and not mass[0, 0, budget:].any()
    assert torch.equal(k.view(S, 8)[:budget], k0.view(S, 8)[best])


def test_captured_and_replayed_in_place(cuda_lib):
    """A captured in-place eviction, replayed on refilled caches, on another stream than the current one."""
    dev = "cuda"
    lens, budget, page = [300, 120], 64, 16
    k, v, table = ref.paged(lens, page, 2, 64, "bf16", 3, stale=0.0)
    m0 = weights(2, 2, table.shape[1] * page, 5)
    kc, vc, mg, tg = k.to(dev), v.to(dev), m0.to(dev), table.to(dev)
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nl, kept = cuda_lib.art_cache_evict(kc, vc, tg, sl, mg, budget, sink=1, recent=9)
    side.synchronize()
    first = [x.clone() for x in (kc, vc, mg, nl, kept)]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        cuda_lib.art_cache_evict(kc, vc, tg, sl, mg, budget, sink=1, recent=9, new_seq_lens=nl, kept=kept)
    for _ in range(2):
        for x, y in ((kc, k), (vc, v), (mg, m0)):
            x.copy_(y)
        nl.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((kc, vc, mg, nl, kept), first))


def test_strided_caches_and_rows(cuda_lib):
    dev = "cuda"
    lens, budget, page = [100, 60], 30, 16
    k, v, table = ref.paged(lens, page, 2, 64, "bf16", 3, stale=0.0)
    m0 = weights(2, 2, table.shape[1] * page, 5)
    a = [x.to(dev) for x in (k, v, table, m0)]
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    nl, kept = cuda_lib.art_cache_evict(a[0], a[1], a[2], sl, a[3], budget, sink=1, recent=3)
    kg = torch.empty(k.shape[0], page, 2, 72, dtype=k.dtype, device=dev).permute(0, 2, 1, 3)[..., :64].copy_(k)
    vg = torch.empty(v.shape[0], 3, page, 64, dtype=v.dtype, device=dev)[:, 1:].copy_(v)
    mg = torch.full((2, 3, m0.shape[2] + 5), 6.0, device=dev)
    mg[:, :2, :m0.shape[2]] = m0.to(dev)
    nl2 = torch.empty(2, dtype=torch.int32, device=dev)
    kp2 = torch.full((2, 2, budget + 4), -5, dtype=torch.int32, device=dev)
    cuda_lib.art_cache_evict(kg, vg, a[2], sl, mg[:, :2, :m0.shape[2]], budget, sink=1, recent=3, new_seq_lens=nl2,
                             kept=kp2[..., :budget])
    torch.cuda.synchronize()
    assert torch.equal(kp2[..., :budget], kept) and torch.equal(nl, nl2) and bool((kp2[..., budget:] == -5).all())
    assert torch.equal(kg, a[0]) and torch.equal(vg, a[1]) and torch.equal(mg[:, :2, :m0.shape[2]], a[3])
    assert bool((mg[:, 2] == 6.0).all()) and bool((mg[..., m0.shape[2]:] == 6.0).all())


@pytest.mark.parametrize("lens", [(3, 1, 33), (130, 127, 129), (9001, 8190, 4099), (20003, 37, 16385)])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_weights_on_any_boundary(cuda_lib, lens, offset):
    """Rows of weights on every 4-byte boundary, ending inside a vector, with
    other numbers right before and behind them."""
    dev, page, Hkv, d = "cuda", 5, 3, 8
    budget = max(lens) // 3 + 1
    k, v, table = ref.paged(list(lens), page, Hkv, d, "bf16", 3, stale=0.0)
    S = table.shape[1] * page
    m0 = weights(len(lens), Hkv, S, offset)
    base = torch.full((len(lens), Hkv, S + 4 + offset), math.inf, device=dev)
    mass = base[..., offset:offset + S].copy_(m0)
    want = [ref.evict_kept(m0[b, h].tolist(), n, budget, 1, 2) for b, n in enumerate(lens) for h in range(Hkv)]
    nl, kept = cuda_lib.art_cache_evict(k.to(dev), v.to(dev), table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                                        mass, budget, sink=1, recent=2)
    torch.cuda.synchronize()
    for row, w, m, src in zip(kept.flatten(0, 1).cpu(), want, mass.flatten(0, 1).cpu(), m0.flatten(0, 1)):
        assert row.tolist() == w + [-1] * (budget - len(w))
        assert torch.equal(m[:len(w)], src[torch.tensor(w, dtype=torch.long)]) and bool((m[len(w):] == 0).all())
    assert bool((base[..., :offset] == math.inf).all()) and bool((base[..., offset + S:] == math.inf).all())


def test_threads_with_sequences_of_different_lengths(cuda_lib):
    """Calls from several host threads at once, on streams of their own."""
    import threading
    dev, page, failed = "cuda", 16, []

    def work(seed, L):
        try:
            stream = torch.cuda.Stream()
            k, v, table = ref.paged([L], page, 1, 8, "bf16", seed, stale=0.0)
            m0 = weights(1, 1, table.shape[1] * page, seed)
            want = ref.evict_kept(m0[0, 0].tolist(), L, L // 2, 1, 1)
            with torch.cuda.stream(stream):
                kc, vc, tb, sl = k.to(dev), v.to(dev), table.to(dev), torch.tensor([L], dtype=torch.int32, device=dev)
                for _ in range(200):
                    nl, kept = cuda_lib.art_cache_evict(kc, vc, tb, sl, m0.to(dev), L // 2, sink=1, recent=1)
            stream.synchronize()
            assert kept[0, 0].tolist() == want
        except Exception as e:                  # noqa: BLE001 (told to the main thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i, L)) for i, L in enumerate((40000, 300, 12000, 8000, 33000, 7000))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_bad_pages_and_long_sequences_are_reported(cuda_lib):
    dev = "cuda"
    lens, budget, page = [64, 64], 32, 16
    k, v, table = ref.paged(lens, page, 1, 64, "bf16", 3, stale=0.0)
    m = torch.zeros(2, 1, 64)
    m[:, :, 32:] = 1.0                       # the last two pages stay
    bad = table.clone()
    bad[0, 3] = -2
    kc, vc = k.to(dev), v.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    cuda_lib.art_cache_evict(kc, vc, bad.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), m.to(dev), budget,
                             device_status=status)
    torch.cuda.synchronize()
    assert int(status) == -8
    want = k.clone()
    want[table[0, 0].long()] = k[table[0, 2].long()]         # its page 3 cannot be read: rows 16.. stay
    for i in (0, 1):
        want[table[1, i].long()] = k[table[1, i + 2].long()]
    assert torch.equal(kc.cpu(), want)
    status.zero_()
    nl, kept = cuda_lib.art_cache_evict(k.to(dev), v.to(dev), table.to(dev), torch.tensor([64, 65], dtype=torch.int32,
                                                                                          device=dev), m.to(dev), budget,
                                        device_status=status)
    torch.cuda.synchronize()
    assert int(status) == -8 and nl.tolist() == [32, 32] and kept[1, 0].tolist() == list(range(32, 64))


def test_a_copy_of_the_own_table_is_reported(cuda_lib):
    """The sequence's own pages given as new ones by a copy of its table: reported, nothing moved; the table itself
    (or its first columns) means in place."""
    dev = "cuda"
    k, v, table = ref.paged([64], 16, 1, 64, "bf16", 3, stale=0.0)
    m = torch.arange(64.0).view(1, 1, 64)
    sl = torch.tensor([64], dtype=torch.int32, device=dev)
    tg = table.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kc, vc = k.to(dev), v.to(dev)
    cuda_lib.art_cache_evict(kc, vc, tg, sl, m.to(dev), 32, new_page_table=tg.clone(), device_status=status)
    torch.cuda.synchronize()
    assert int(status) == -8 and torch.equal(kc.cpu(), k) and torch.equal(vc.cpu(), v)
    status.zero_()
    cuda_lib.art_cache_evict(kc, vc, tg, sl, m.to(dev), 32, new_page_table=tg[:, :2], device_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(ref.rows(kc.cpu(), table, 0, 0, 32), ref.rows(k, table, 0, 0, 64)[32:])


@pytest.mark.parametrize("budget", [4990, 2500, 300])
def test_long_rows_slide_in_place(cuda_lib, budget):
    """Several CTAs on one unit's rows: most stay, half, few."""
    run(cuda_lib, [5000, 17], budget, sink=3, recent=min(100, budget // 4), Hkv=1, d=128, page=64, in_place=True, seed=budget)


def test_offsets_past_32_bits(cuda_lib):
    dev = "cuda"
    page, Hkv, d = 64, 8, 128
    pages = 2 ** 31 // (page * Hkv * d) + 9
    kc = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device=dev)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=dev)
    kc[-2:] = torch.randn(2, Hkv, page, d, device=dev).to(torch.bfloat16)
    old = kc[-2:].clone()
    mass = torch.arange(128, dtype=torch.float32, device=dev).expand(1, Hkv, 128).contiguous()
    cuda_lib.art_cache_evict(kc, kc[...], table, torch.tensor([128], dtype=torch.int32, device=dev), mass, 64)
    torch.cuda.synchronize()
    assert torch.equal(kc[-1], old[0])


# (sequences, heads, columns) whose selection runs on so many CTAs a unit
CLUSTERS = {1: (3, 2, 4000), 2: (35, 2, 40000), 3: (20, 2, 40000), 4: (3, 1, 15008), 5: (3, 1, 18000), 6: (3, 1, 22000),
            7: (3, 1, 26000), 8: (3, 1, 30000)}


@PLACES
@pytest.mark.parametrize("kind", ["ties", "equal", "distinct"])
@pytest.mark.parametrize("ctas", CLUSTERS)
def test_every_cluster_size(cuda_lib, in_place, kind, ctas):
    """One sequence that fills the table and short ones beside it, on 1 to 8 CTAs a unit (the size asked of the library);
    the last kept token among ties that several CTAs hold, among tokens all equal, and with no ties."""
    B, Hkv, S = CLUSTERS[ctas]
    page, d = 16, 8
    lens = [S] + [(S // 3 + 37, 1, 700, 0, 33)[i % 5] if i < 5 else 40 + 31 * i for i in range(B - 1)]
    budget = S // 3
    p = cuda_lib.ArtEvictParams()
    fake = lambda shape, dt: cuda_lib.descriptor(torch.empty(1, dtype=dt, device="cuda").expand(shape))   # noqa: E731

    def dense(shape, dt):
        t, step = fake(shape, dt), 1
        for i in reversed(range(len(shape))):
            t.stride[i] = step
            step *= shape[i]
        return t

    i32, f32, blocks = torch.int32, torch.float32, S // page
    for name, shape, dt in (("k_cache", (9, Hkv, page, d), torch.bfloat16), ("v_cache", (9, Hkv, page, d), torch.bfloat16),
                            ("page_table", (B, blocks), i32), ("seq_lens", (B,), i32), ("mass", (B, Hkv, S), f32),
                            ("new_seq_lens", (B,), i32), ("kept", (B, Hkv, budget), i32)):
        setattr(p, name, dense(shape, dt))
    p.new_seq_lens.data = p.seq_lens.data + 4096
    p.budget, p.sink, p.recent = budget, 4, 100
    assert cuda_lib.raw_library().art_evict_cluster_size(bytes(p)) == ctas
    mass = weights(B, Hkv, S, ctas, "ties" if kind == "ties" else "distinct")
    if kind == "equal":
        mass.fill_(0.5)
    run(cuda_lib, lens, budget, sink=4, recent=100, Hkv=Hkv, d=d, page=page, width=blocks, in_place=in_place, mass=mass,
        seed=ctas)
